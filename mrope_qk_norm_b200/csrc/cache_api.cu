// cache_api.cu -- C ABI of the paged cache: validation, launch shapes, launch.

#include <atomic>
#include <climits>
#include <cmath>

#include "cache_internal.cuh"

using qkr::api_done;
using qkr::api_fail;

namespace {

struct Bytes {
    uintptr_t lo = 0, hi = 0;
};
Bytes bytes_of(const void *p, __int128 n)
{
    Bytes b;
    if (p && n > 0) {
        b.lo = reinterpret_cast<uintptr_t>(p);
        b.hi = b.lo + (uintptr_t)n;
    }
    return b;
}
bool meet(const Bytes &a, const Bytes &b)
{
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// The rows of a [T, H, D] view: T runs of `width` bytes, `step` apart.
struct Rows {
    const void *base;
    int64_t T, step, width;
    Bytes all() const { return bytes_of(base, (__int128)(T - 1) * step + width); }
};
// Do two views share a byte?  Not if they are column windows of one buffer: the same
// step, and each row of one between rows of the other.
bool meet(const Rows &a, const Rows &b)
{
    if (!meet(a.all(), b.all()))
        return false;
    if (a.step != b.step || a.width > a.step || b.width > b.step)
        return true;
    const int64_t diff = (int64_t)(reinterpret_cast<uintptr_t>(b.base) -
                                   reinterpret_cast<uintptr_t>(a.base)) % a.step;
    const int64_t at = diff < 0 ? diff + a.step : diff;     // b's row from the start of a's
    return at < a.width || at + b.width > a.step;
}
bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

Bytes plane_bytes(const qkr::CachePlane &pl, const qkr::CacheView &c, int64_t row_bytes)
{
    return bytes_of(pl.base, (__int128)(c.n_pages - 1) * pl.ps + (__int128)(c.page_size - 1) * pl.rs +
                                 (__int128)(c.Hkv - 1) * pl.hs + row_bytes);
}

qkr_status check_plane(const char *name, const qkr_cache_plane &in, const qkr_cache_desc &c,
                       int64_t row_bytes, int64_t align, qkr::CachePlane *out)
{
    if (!in.base)
        return api_fail(QKR_ERR_INVALID_ARG, "cache %s is NULL", name);
    if (!aligned(in.base, align))
        return api_fail(QKR_ERR_UNSUPPORTED, "cache %s must be %lld-byte aligned", name,
                        (long long)align);
    const int64_t strides[3] = {in.page_stride, in.row_stride, in.head_stride};
    const int64_t extent[3] = {c.n_pages, c.page_size, c.Hkv};
    int64_t use[3];
    for (int i = 0; i < 3; ++i) {
        use[i] = extent[i] > 1 ? strides[i] : 0;  // the stride of a single row is never used
        if (extent[i] > 1 && strides[i] < row_bytes)
            return api_fail(QKR_ERR_UNSUPPORTED, "cache %s: strides must not make rows overlap",
                            name);
        if (use[i] % align)
            return api_fail(QKR_ERR_UNSUPPORTED, "cache %s: strides must be multiples of %lld bytes",
                            name, (long long)align);
        if (use[i] >= (int64_t)1 << (i < 2 ? 32 : 39))
            return api_fail(QKR_ERR_UNSUPPORTED, "cache %s: page and row strides must be below 2^32 "
                            "bytes, head strides below 2^39", name);
    }
    out->base = static_cast<uint8_t *>(in.base);
    out->ps = use[0];
    out->rs = use[1];
    out->hs = use[2];
    return QKR_OK;
}

qkr_status check_cache_sizes(const qkr_cache_desc *c)
{
    if (!c)
        return api_fail(QKR_ERR_INVALID_ARG, "cache descriptor is NULL");
    if (c->format != QKR_CACHE_BF16 && c->format != QKR_CACHE_Q4)
        return api_fail(QKR_ERR_INVALID_ARG, "unknown cache format %d", c->format);
    if (c->Hkv < 1 || c->Hkv > 65536)
        return api_fail(QKR_ERR_INVALID_ARG, "Hkv must be in [1, 65536]");
    if (c->format == QKR_CACHE_BF16 && (c->D < 8 || c->D > 128 || c->D % 8))
        return api_fail(QKR_ERR_UNSUPPORTED, "head_dim %lld: need a multiple of 8 in [8, 128]",
                        (long long)c->D);
    if (c->format == QKR_CACHE_Q4 && c->D != 64 && c->D != 128)
        return api_fail(QKR_ERR_UNSUPPORTED, "head_dim %lld: a 4-bit cache has 64 or 128",
                        (long long)c->D);
    return QKR_OK;
}

qkr_status check_cache(const qkr_cache_desc *c, qkr::CacheView *v)
{
    qkr_status st = check_cache_sizes(c);
    if (st != QKR_OK)
        return st;
    if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16)
        return api_fail(QKR_ERR_UNSUPPORTED, "page_size %d: need a multiple of 16 in [16, 65536]",
                        c->page_size);
    if (c->n_pages < 1 || c->n_pages > INT_MAX)
        return api_fail(QKR_ERR_INVALID_ARG, "n_pages must be in [1, 2^31)");
    const bool q4 = c->format == QKR_CACHE_Q4;
    const int64_t row = q4 ? c->D / 2 : c->D * 2;
    *v = qkr::CacheView{};
    if ((st = check_plane("k", c->k, *c, row, 16, &v->k)) != QKR_OK ||
        (st = check_plane("v", c->v, *c, row, 16, &v->v)) != QKR_OK)
        return st;
    if (q4 && ((st = check_plane("k_scale", c->k_scale, *c, c->D / 16, c->D / 16, &v->ks)) != QKR_OK ||
               (st = check_plane("v_scale", c->v_scale, *c, c->D / 16, c->D / 16, &v->vs)) != QKR_OK))
        return st;
    v->page_size = c->page_size;
    v->n_pages = (int)c->n_pages;
    v->Hkv = (int)c->Hkv;
    v->D = (int)c->D;
    return QKR_OK;
}

bool meets_cache(const Bytes &b, const qkr::CacheView &v, bool q4)
{
    const int64_t row = q4 ? v.D / 2 : v.D * 2;
    return meet(b, plane_bytes(v.k, v, row)) || meet(b, plane_bytes(v.v, v, row)) ||
           (q4 && (meet(b, plane_bytes(v.ks, v, v.D / 16)) ||
                   meet(b, plane_bytes(v.vs, v, v.D / 16))));
}

// out, lse and the workspace against each other, the inputs (q is the first) and the
// cache; out and q row by row.
qkr_status check_overlap(const Bytes (&written)[3], const Bytes (&read)[4], const Rows &out,
                         const Rows &q, const qkr::CacheView &view, bool q4)
{
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 4; ++j)
            if (i == 0 && j == 0 ? meet(out, q) : meet(written[i], read[j]))
                return api_fail(QKR_ERR_UNSUPPORTED,
                                "out, lse and workspace must not overlap an input");
        for (int j = 0; j < i; ++j)
            if (meet(written[i], written[j]))
                return api_fail(QKR_ERR_UNSUPPORTED, "out, lse and workspace must not overlap");
        if (meets_cache(written[i], view, q4))
            return api_fail(QKR_ERR_UNSUPPORTED,
                            "out, lse and workspace must not overlap the cache");
    }
    return QKR_OK;
}

qkr_status cuda_fail(cudaError_t e, const char *what)
{
    return api_fail(QKR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// What a call needs to know of the current device; asked of the driver once.
constexpr int kMaxDevices = 64;
struct Device {
    std::atomic<int> sms{0};
    std::atomic<unsigned *> status{nullptr};
};
Device g_devices[kMaxDevices];

// Kernels allowed their dynamic shared memory, a bit a device.  Nothing here
// allocates or throws; two threads that ask at once both ask the driver.
constexpr int kMaxKernels = 64;
struct SmemSeen {
    std::atomic<const void *> fn{nullptr};
    std::atomic<uint64_t> devices{0};
};
SmemSeen g_smem[kMaxKernels];

qkr_status current_device(int *sms, unsigned **status)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    if (dev < 0 || dev >= kMaxDevices)
        return api_fail(QKR_ERR_UNSUPPORTED, "device %d: at most %d devices", dev, kMaxDevices);
    Device &d = g_devices[dev];
    *sms = d.sms.load(std::memory_order_relaxed);
    if (*sms == 0) {
        e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return cuda_fail(e, "device query");
        d.sms.store(*sms, std::memory_order_relaxed);
    }
    *status = d.status.load(std::memory_order_relaxed);
    if (!*status) {
        e = qkr::device_status_address(status);
        if (e != cudaSuccess)
            return cuda_fail(e, "status word");
        d.status.store(*status, std::memory_order_relaxed);
    }
    return QKR_OK;
}

// Sizes every cache_attention launch shape follows from.
struct Sizes {
    int64_t T, Hq, Hkv, D, B, max_q, max_len, window, n_sink;
    int q4;
};

qkr_status check_sizes(Sizes &s)
{
    if (s.T < 0 || s.B < 0 || s.max_q < 0 || s.max_len < 0)
        return api_fail(QKR_ERR_INVALID_ARG, "T, B, max_q and max_len must be >= 0");
    if (s.Hq < 1 || s.Hq % s.Hkv || s.Hq > 65536)
        return api_fail(QKR_ERR_INVALID_ARG, "Hq (%lld) must be a multiple of Hkv (%lld), at most "
                        "65536", (long long)s.Hq, (long long)s.Hkv);
    if (s.T > INT_MAX || s.T * s.Hq > INT_MAX || s.B > (1 << 16) || s.max_len > (1 << 29))
        return api_fail(QKR_ERR_UNSUPPORTED, "need T * Hq < 2^31, B <= 2^16, max_len <= 2^29");
    if (s.window < 0 || s.n_sink < 0)
        return api_fail(QKR_ERR_INVALID_ARG, "window and n_sink must be >= 0");
    if (s.max_q > s.T)
        s.max_q = s.T;
    if (s.window >= s.max_len)
        s.window = 0;  // nothing is ever that far back
    if (s.n_sink > s.max_len)
        s.n_sink = s.max_len;
    return QKR_OK;
}

// How a call runs: the block and split of each kernel that takes part.
struct Plan {
    bool rows = false, tiles = false;
    qkr::AttnParams pr = {}, pt = {};
    int64_t ws_bytes = 0;
    unsigned *status = nullptr;
};

// Blocks of a launch that serves sequences of up to `hi` rows, and the tiles
// a block can have.
int64_t blocks(const Sizes &s, int block_rows, int tile, int64_t lo, int64_t hi,
               qkr::AttnParams *p)
{
    const int64_t G = s.Hq / s.Hkv;
    p->rows = block_rows;
    p->rows_lo = (int)lo;
    p->rows_hi = (int)hi;
    p->tile = tile;
    const int64_t most = s.max_q * G < hi ? s.max_q * G : hi;
    const int64_t per_seq = (most + block_rows - 1) / block_rows;
    const int64_t by_total = s.T * G / block_rows + s.B;
    p->direct = s.B * per_seq <= by_total;
    p->blocks_max = (int)per_seq;
    p->n_blocks = p->direct ? s.B * per_seq : by_total;
    // the window and the sinks may each start inside a tile
    int64_t keys = s.max_len;
    if (s.window && s.window + s.n_sink + block_rows / G + 1 < keys)
        keys = s.window + s.n_sink + block_rows / G + 1;
    return keys / tile + (s.window ? 3 : 1);
}

// Cuts the axis into parts of `split` tiles, 1024 at most.
void cut(const Sizes &s, int64_t tiles, int64_t split, qkr::AttnParams *p, int64_t *ws)
{
    if (tiles > split * 1024)
        split = (tiles + 1023) / 1024;
    const int64_t n = (tiles + split - 1) / split;
    p->split_tiles = (int)split;
    p->nsplit = (int)n;
    const int64_t need = n > 1 ? n * s.T * s.Hq * (s.D + 2) * 4 : 0;
    if (need > *ws)
        *ws = need;
}

// Sequences of up to kFewRows rows go to the rows kernel, longer ones to the
// tiles kernel; both run where a call can hold both kinds.  One sequence, or
// as many new tokens as every sequence having max_q would make, is one kind.
constexpr int64_t kFewRows = 16;

qkr_status make_plan(const Sizes &s, int64_t page_size, Plan *plan)
{
    int sms = 0;
    qkr_status st = current_device(&sms, &plan->status);
    if (st != QKR_OK)
        return st;
    const int64_t G = s.Hq / s.Hkv, most = s.max_q * G;
    plan->tiles = most > kFewRows;
    plan->rows = !plan->tiles || (s.B > 1 && s.T < s.B * s.max_q && G <= kFewRows);
    if (plan->rows) {
        qkr::AttnParams &p = plan->pr;
        const int64_t cap = plan->tiles ? kFewRows : INT_MAX;
        int shift = 6;
        while (page_size % ((int64_t)1 << shift))
            --shift;
        p.tile_shift = shift;
        const int64_t tiles = blocks(s, (most < cap ? most : cap) <= 8 ? 8 : 16, 1 << shift, 0, cap, &p);
        const int64_t keys = tiles << shift;
        const int64_t items = p.n_blocks * s.Hkv;   // one block a sequence
        const int64_t slots = (int64_t)sms * qkr::attn_rows_resident(s.D, p.rows, s.q4);
        // A cluster a block, as large as leaves a warp 32 keys and the clusters
        // room, where a warp then has at most 96 keys.  Else even shares, of no
        // less than 128 keys; a block counts for 128 keys more, 512 in 4 bits, whose
        // keys take less time (ragged decode batches, bf16: 88 us at 0, 72 at 128, 74
        // at 512; 4 bits: 60 at 128, 53 at 512).
        p.nsplit = 1;
        int64_t size = 1;
        while (size < 8 && keys > size * 128 && items * size * 2 <= slots)
            size *= 2;
        if (keys <= size * 4 * 96 && items * size <= 2 * slots) {
            p.cluster = (int)size;
        } else {
            p.ctas = (int)slots;
            p.split_tiles = 128 >> shift;
            p.piece_cost = (s.q4 ? 512 : 128) >> shift;
            plan->ws_bytes = slots * (2 * p.rows * (s.D + 2) * 4 + (int64_t)sizeof(qkr::AttnSpan));
        }
    }
    if (plan->tiles) {
        qkr::AttnParams &p = plan->pt;
        p.tile_shift = 7;
        const int64_t tiles = blocks(s, 256, 128, plan->rows ? kFewRows : 0, INT_MAX, &p);
        // Parts of a block's keys: the number that takes the fewest rounds over the
        // SMs times what a CTA then does, its tiles and some 5 tiles' time of setting
        // up and writing out (20 of 3400 clocks a tile); joining parts costs 3 more.
        // A sequence's last block is counted half (four chunks of 300 to 512 tokens
        // on 8192 cached in 4 bits: 142 us in 3 parts, 129 whole; 106 since).
        const int64_t most_items = p.n_blocks * s.Hkv;
        int64_t items = (s.T * G / 256 + (s.B + 1) / 2) * s.Hkv;
        if (items > most_items)
            items = most_items;
        if (items < 1)
            items = 1;
        int64_t best = 1, best_cost = INT64_MAX;
        // (with two rounds or more the blocks' own lengths even out)
        for (int64_t n = 1; n <= (items >= 2 * sms ? 1 : 64) && n <= tiles; ++n) {
            const int64_t rounds = (items * n + sms - 1) / sms;
            const int64_t cost = rounds * ((tiles + n - 1) / n + 5) + (n > 1 ? 3 : 0);
            if (cost < best_cost) {
                best_cost = cost;
                best = n;
            }
        }
        cut(s, tiles, (tiles + best - 1) / best, &p, &plan->ws_bytes);
    }
    if ((plan->rows && plan->pr.n_blocks * s.Hkv > INT_MAX / 256) ||
        (plan->tiles && plan->pt.n_blocks * s.Hkv * plan->pt.nsplit > INT_MAX / 256))
        return api_fail(QKR_ERR_UNSUPPORTED, "the call needs more blocks than a launch takes");
    return QKR_OK;
}

}  // namespace

cudaError_t qkr::allow_smem(const void *fn, int bytes)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    SmemSeen *seen = nullptr;
    for (SmemSeen &k : g_smem) {
        const void *have = nullptr;
        if (k.fn.compare_exchange_strong(have, fn) || have == fn) {
            seen = &k;
            break;
        }
    }
    const uint64_t bit = dev >= 0 && dev < kMaxDevices ? (uint64_t)1 << dev : 0;
    if (seen && (seen->devices.load() & bit))
        return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && seen)
        seen->devices.fetch_or(bit);
    return e;
}

extern "C" {

qkr_status cache_attention_workspace(const qkr_cache_desc *cache, int64_t T, int64_t Hq,
                                     int64_t B, int64_t max_q, int64_t max_len, int64_t window,
                                     int64_t n_sink, int64_t *bytes)
{
    if (!bytes)
        return api_fail(QKR_ERR_INVALID_ARG, "bytes is NULL");
    qkr_status st = check_cache_sizes(cache);
    if (st != QKR_OK)
        return st;
    Sizes s = {T, Hq, cache->Hkv, cache->D, B, max_q, max_len, window, n_sink,
               cache->format == QKR_CACHE_Q4};
    if ((st = check_sizes(s)) != QKR_OK)
        return st;
    if (cache->page_size < 16 || cache->page_size > 65536 || cache->page_size % 16)
        return api_fail(QKR_ERR_UNSUPPORTED, "page_size %d: need a multiple of 16 in [16, 65536]",
                        cache->page_size);
    Plan plan;
    if (s.T && s.B && s.max_q && (st = make_plan(s, cache->page_size, &plan)) != QKR_OK)
        return st;
    *bytes = plan.ws_bytes;
    return api_done(qkr::LaunchRecord());
}

qkr_status cache_attention(void *stream, const qkr_cache_desc *cache, const void *q, void *out,
                           float *lse, int64_t T, int64_t Hq, int64_t q_tok_stride,
                           int64_t q_head_stride, int64_t out_tok_stride,
                           const int32_t *page_table, int64_t table_stride, const int32_t *lens,
                           const int32_t *cu_q, int64_t B, int64_t max_q, int64_t max_len,
                           float scale, int64_t window, int64_t n_sink, void *workspace,
                           int64_t workspace_bytes)
{
    qkr::CacheView view;
    qkr_status st = check_cache(cache, &view);
    if (st != QKR_OK)
        return st;
    const bool q4 = cache->format == QKR_CACHE_Q4;
    Sizes s = {T, Hq, cache->Hkv, cache->D, B, max_q, max_len, window, n_sink, q4};
    if ((st = check_sizes(s)) != QKR_OK)
        return st;
    // the softmax works in powers of two
    const float scale_log2 = (float)((double)scale * 1.4426950408889634);
    if (!std::isfinite(scale_log2))
        return api_fail(QKR_ERR_INVALID_ARG, "scale must be finite, at most 2^127 in magnitude");
    if (s.T == 0 || s.B == 0 || s.max_q == 0)
        return api_done(qkr::LaunchRecord());
    if (!q || !out || !lens || !cu_q || (s.max_len && !page_table))
        return api_fail(QKR_ERR_INVALID_ARG, "q, out, page_table, lens and cu_q must be non-NULL");
    if (!aligned(q, 16) || !aligned(out, 16))
        return api_fail(QKR_ERR_UNSUPPORTED, "q and out must be 16-byte aligned");
    if (!aligned(lens, 4) || !aligned(cu_q, 4) || !aligned(page_table, 4) || !aligned(lse, 4))
        return api_fail(QKR_ERR_UNSUPPORTED, "page_table, lens, cu_q and lse must be 4-byte aligned");
    if (s.T == 1) {     // the stride of a single token is never used
        q_tok_stride = 0;
        out_tok_stride = s.Hq * s.D;
    }
    if (q_head_stride < s.D || q_head_stride % 8 || (s.T > 1 && q_tok_stride <= 0) ||
        q_tok_stride % 8 || out_tok_stride < s.Hq * s.D || out_tok_stride % 8)
        return api_fail(QKR_ERR_UNSUPPORTED,
                        "strides must be multiples of 8 elements, heads must not overlap and out "
                        "rows must hold a token's heads");
    const int64_t far = (int64_t)1 << 45;
    if (q_tok_stride > far / s.T || q_head_stride > far / s.Hq || out_tok_stride > far / s.T)
        return api_fail(QKR_ERR_INVALID_ARG, "a view exceeds the address range");
    if (table_stride < 0 || table_stride > INT_MAX || s.max_len > table_stride * view.page_size)
        return api_fail(QKR_ERR_INVALID_ARG,
                        "max_len (%lld) exceeds the page table: %lld pages of %d tokens",
                        (long long)s.max_len, (long long)table_stride, view.page_size);

    const Rows q_rows = {q, s.T, 2 * q_tok_stride, 2 * ((s.Hq - 1) * q_head_stride + s.D)};
    const Rows out_rows = {out, s.T, 2 * out_tok_stride, 2 * s.Hq * s.D};
    const Bytes read[4] = {
        q_rows.all(),
        bytes_of(page_table, (__int128)4 * s.B * table_stride), bytes_of(lens, 4 * s.B),
        bytes_of(cu_q, 4 * (s.B + 1))};
    Bytes written[3] = {out_rows.all(), bytes_of(lse, 4 * s.T * s.Hq), Bytes()};
    if ((st = check_overlap(written, read, out_rows, q_rows, view, q4)) != QKR_OK)
        return st;
    Plan plan;
    if ((st = make_plan(s, view.page_size, &plan)) != QKR_OK)
        return st;
    if (plan.ws_bytes > 0) {
        if (!workspace || workspace_bytes < plan.ws_bytes)
            return api_fail(QKR_ERR_INVALID_ARG, "workspace of %lld bytes, needs %lld",
                            (long long)(workspace ? workspace_bytes : 0), (long long)plan.ws_bytes);
        if (!aligned(workspace, 16))
            return api_fail(QKR_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
        written[2] = bytes_of(workspace, plan.ws_bytes);
        if ((st = check_overlap(written, read, out_rows, q_rows, view, q4)) != QKR_OK)
            return st;
    }

    cudaError_t e;
    qkr::LaunchRecord rec;
    for (int which = 0; which < 2; ++which) {
        if (!(which ? plan.tiles : plan.rows))
            continue;
        qkr::AttnParams &p = which ? plan.pt : plan.pr;
        p.c = view;
        p.q = static_cast<const __nv_bfloat16 *>(q);
        p.q_ts = q_tok_stride;
        p.q_hs = q_head_stride;
        p.out = static_cast<__nv_bfloat16 *>(out);
        p.o_ts = out_tok_stride;
        p.lse = lse;
        p.table = page_table;
        p.table_stride = table_stride;
        p.lens = lens;
        p.cu = cu_q;
        p.T = s.T;
        p.B = (int)s.B;
        p.Hq = (int)s.Hq;
        p.G = (int)(s.Hq / s.Hkv);
        p.max_q = (int)s.max_q;
        p.max_len = (int)s.max_len;
        p.window = (int)s.window;
        p.n_sink = (int)s.n_sink;
        p.scale_log2 = scale_log2;
        p.ws_o = static_cast<float *>(workspace);
        const int64_t kept = p.ctas ? 2 * (int64_t)p.ctas * p.rows : (int64_t)p.nsplit * s.T * s.Hq;
        p.ws_ml = reinterpret_cast<float2 *>(p.ws_o + kept * s.D);
        p.ws_span = reinterpret_cast<qkr::AttnSpan *>(p.ws_ml + kept);
        if (q4) {
            p.dense_scales = 1;
            for (const qkr::CachePlane *pl : {&view.ks, &view.vs})
                if (pl->rs != s.D / 16 || pl->hs % 16 || pl->ps % 16 || !aligned(pl->base, 16))
                    p.dense_scales = 0;
        }
        const uint64_t page_tiles = view.page_size >> p.tile_shift;
        if (!which)
            p.page_recip = (((uint64_t)1 << 38) + page_tiles - 1) / page_tiles;
        p.status = plan.status;
        const cudaStream_t cs = static_cast<cudaStream_t>(stream);
        const int64_t launches = rec.launches;
        rec = qkr::LaunchRecord();      // the last kernel's own shape, all launches
        rec.launches = launches;
        if (which && p.scale_log2 == 0.f)
            p.scale_log2 = 0x1p-149f;  // masked scores are -infinity times the scale, and
                                       // any finite score times this is below 2^-21
        e = which ? qkr::launch_attn_tiles(p, q4, cs, &rec) : qkr::launch_attn_rows(p, q4, cs, &rec);
        if (e != cudaSuccess)
            return cuda_fail(e, "cache attention launch");
        if (which && p.nsplit > 1) {
            e = qkr::launch_attn_join(p, cs);
            if (e != cudaSuccess)
                return cuda_fail(e, "cache attention join launch");
            rec.launches += 1;
        }
    }
    return api_done(rec);
}

static qkr_status rows_q4(void *stream, const qkr_cache_desc *cache, const void *k, const void *v,
                          const int64_t *row_idx, int64_t T, int64_t k_ts, int64_t v_ts, bool set)
{
    qkr::CacheView view;
    qkr_status st = check_cache(cache, &view);
    if (st != QKR_OK)
        return st;
    if (cache->format != QKR_CACHE_Q4)
        return api_fail(QKR_ERR_INVALID_ARG, "the cache must be QKR_CACHE_Q4");
    if (T < 0)
        return api_fail(QKR_ERR_INVALID_ARG, "T must be >= 0");
    if (T == 0)
        return api_done(qkr::LaunchRecord());
    if (T > INT_MAX || T * cache->Hkv > ((int64_t)1 << 30))
        return api_fail(QKR_ERR_UNSUPPORTED, "need T * Hkv <= 2^30");
    if (!k || !v || !row_idx)
        return api_fail(QKR_ERR_INVALID_ARG, "k, v and row_idx must be non-NULL");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(row_idx, 8))
        return api_fail(QKR_ERR_UNSUPPORTED, "k and v must be 16-byte aligned, row_idx 8-byte");
    const int64_t row = cache->Hkv * cache->D;
    if (k_ts < row || v_ts < row || k_ts % 8 || v_ts % 8 || k_ts > ((int64_t)1 << 45) / T ||
        v_ts > ((int64_t)1 << 45) / T)
        return api_fail(QKR_ERR_UNSUPPORTED,
                        "token strides must be multiples of 8 and hold a token's heads");
    const Rows rk = {k, T, 2 * k_ts, 2 * row}, rv = {v, T, 2 * v_ts, 2 * row};
    const Bytes bk = rk.all(), bv = rv.all(), bi = bytes_of(row_idx, 8 * T);
    if (meets_cache(bk, view, true) || meets_cache(bv, view, true) || meets_cache(bi, view, true))
        return api_fail(QKR_ERR_UNSUPPORTED, "k, v and row_idx must not overlap the cache");
    if (!set && (meet(rk, rv) || meet(bk, bi) || meet(bv, bi)))
        return api_fail(QKR_ERR_UNSUPPORTED, "k_out, v_out and row_idx must not overlap");
    unsigned *status = nullptr;
    int sms = 0;
    if ((st = current_device(&sms, &status)) != QKR_OK)
        return st;
    cudaError_t e;
    qkr::LaunchRecord rec;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    auto *kb = static_cast<__nv_bfloat16 *>(const_cast<void *>(k));
    auto *vb = static_cast<__nv_bfloat16 *>(const_cast<void *>(v));
    e = set ? qkr::launch_set_rows_q4(view, kb, vb, row_idx, T, k_ts, v_ts, status, cs, &rec)
            : qkr::launch_get_rows_q4(view, kb, vb, row_idx, T, k_ts, v_ts, status, cs, &rec);
    return e == cudaSuccess ? api_done(rec) : cuda_fail(e, set ? "set rows launch" : "get rows launch");
}

qkr_status cache_set_rows_q4(void *stream, const qkr_cache_desc *cache, const void *k,
                             const void *v, const int64_t *row_idx, int64_t T,
                             int64_t k_tok_stride, int64_t v_tok_stride)
{
    return rows_q4(stream, cache, k, v, row_idx, T, k_tok_stride, v_tok_stride, true);
}

qkr_status cache_get_rows_q4(void *stream, const qkr_cache_desc *cache, void *k_out, void *v_out,
                             const int64_t *row_idx, int64_t T, int64_t k_tok_stride,
                             int64_t v_tok_stride)
{
    return rows_q4(stream, cache, k_out, v_out, row_idx, T, k_tok_stride, v_tok_stride, false);
}

}  // extern "C"
