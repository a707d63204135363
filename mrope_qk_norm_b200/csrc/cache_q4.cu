// cache_q4.cu -- rows into and out of the 4-bit cache.
//
// Four lanes share a head row of K or V; lane c holds the elements 8c .. 8c+7
// of each group of 32, so a group's extremes are two shuffles away and the
// lane's codes of all groups are D/8 consecutive bytes of the row: for K the
// words (c, w), for V the half words (2c, w) and (2c + 1, w).  One 16-byte (D =
// 128) store a lane, every row in whole 32-byte sectors.
//
// s = e / -8 rounded up to 5 significant bits is bit arithmetic on fp32, and the
// codes are those of the exact quotient (code_of), so equal inputs give equal codes
// on any machine.

#include "cache_attn.cuh"

namespace qkr {
namespace {

constexpr int kThreads = 128;

struct RowsQ4 {
    CacheView c;
    __nv_bfloat16 *x[2];      // K, V rows outside the cache
    int64_t ts[2];
    const int64_t *rows;
    int64_t T;
    unsigned *status;
};

// The head row a thread works on: K or V, token, head, and its place in the cache.
struct Where {
    int which, head, lane4;
    int64_t t;
    int64_t page;
    int row;
    bool inside;
};

// (32-bit divisions: T * Hkv <= 2^30, and few caches have 2^32 rows.)
__device__ __forceinline__ bool locate(const RowsQ4 &p, Where *w)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    w->lane4 = (int)(i & 3);
    const uint32_t r = (uint32_t)(i >> 2), H = (uint32_t)p.c.Hkv, th = r / H;
    w->head = (int)(r - th * H);
    w->which = (int)(th & 1);
    w->t = th >> 1;
    if (w->t >= p.T)
        return false;
    const int64_t at = p.rows[w->t];
    const uint32_t ps = (uint32_t)p.c.page_size;
    w->inside = at >= 0 && at < (int64_t)p.c.n_pages * p.c.page_size;
    if ((uint64_t)at >> 32 == 0) {
        w->page = (uint32_t)at / ps;
        w->row = (int)((uint32_t)at % ps);
    } else {
        w->page = at / p.c.page_size;
        w->row = (int)(at % p.c.page_size);
    }
    if (!w->inside && w->lane4 == 0 && w->head == 0)
        atomicOr(p.status, kStatusRow);
    return true;
}

__device__ __forceinline__ uint8_t *place(const CachePlane &pl, const Where &w)
{
    return pl.base + w.page * pl.ps + w.row * pl.rs + w.head * pl.hs;
}

// The scale of a group with extremes hi and lo, its magnitude at most 31 * 2^120
// (the largest of 5 bits whose eightfold is a finite bf16 number).  The carry rounds a
// subnormal e up to a multiple of 2^-130, with fewer significant bits: 3 bits times it are
// still a multiple of 2^-133, so a bf16 number.
__device__ __forceinline__ float group_scale(float hi, float lo)
{
    const float e = (-lo >= hi ? lo : hi) * -0.125f;
    const float s = __uint_as_float((__float_as_uint(e) + 0x7ffffu) & ~0x7ffffu);
    return fminf(fmaxf(s, -31.f * 0x1p120f), 31.f * 0x1p120f);
}

// min(rint(x / s), 7) + 8 from r = 1/s rounded (never below 0: s is rounded up, or
// at its largest still above x / 8.5).  x r is within 2^-21 of x / s; adding 1536
// rounds it to a multiple of 2^-13.  x has 8 significant bits and s 5, so a quotient
// that is not half way between two codes is at least 2^-5 / 62 from it, and one
// that is becomes exactly that: the rounding below sees the true side and the true
// ties (to even).  It leaves the code in the low bits of 1.5 * 2^23 + code.
__device__ __forceinline__ uint32_t code_of(float x, float r)
{
    const float t = fminf(fmaf(x, r, 1536.f), 1543.f);
    return __float_as_uint(t + 12581384.f) & 15u;      // 12582912 + 8 - 1536
}

template <int D>
__global__ void __launch_bounds__(kThreads) set_rows_q4_kernel(const __grid_constant__ RowsQ4 p)
{
    constexpr int GR = D / 32;
    pdl_wait();
    pdl_trigger();
    Where at;
    const bool live = locate(p, &at);
    uint4 v[GR];
    if (live) {
        const __nv_bfloat16 *src = p.x[at.which] + at.t * p.ts[at.which] + at.head * D + 8 * at.lane4;
#pragma unroll
        for (int w = 0; w < GR; ++w)
            v[w] = ld_stream(src + 32 * w);
    } else {
#pragma unroll
        for (int w = 0; w < GR; ++w)
            v[w] = make_uint4(0, 0, 0, 0);
    }
    uint32_t code[GR];       // nibble i: element 8c + i of group w
    uint32_t scale[GR / 2];  // bf16 pairs
#pragma unroll
    for (int w = 0; w < GR; ++w) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v[w]);
        const __nv_bfloat162 h2 = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        const __nv_bfloat162 l2 = __hmin2(__hmin2(h[0], h[1]), __hmin2(h[2], h[3]));
        float hi = fmaxf(__low2float(h2), __high2float(h2));
        float lo = fminf(__low2float(l2), __high2float(l2));
        uint32_t top = __vmaxu2(__vmaxu2(v[w].x & 0x7fff7fffu, v[w].y & 0x7fff7fffu),
                                __vmaxu2(v[w].z & 0x7fff7fffu, v[w].w & 0x7fff7fffu));
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        const bool bad = (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u;   // inf or NaN
        const float s = group_scale(hi, lo);
        float f[8];
        unpack8(v[w], f);
        uint32_t q = 0;
        if (bad || s == 0.f) {
            q = 0x88888888u;
        } else if (fabsf(s) >= 0x1p-60f) {
            const float r = __frcp_rn(s);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q |= code_of(f[i], r) << (4 * i);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = fminf(fmaxf(rintf(__fdiv_rn(f[i], s)), -8.f), 7.f);
                q |= (uint32_t)((int)c + 8) << (4 * i);
            }
        }
        code[w] = q;
        const uint32_t bits = bad ? 0x7fc0u : __float_as_uint(s) >> 16;
        if (w & 1)
            scale[w / 2] |= bits << 16;
        else
            scale[w / 2] = bits;
    }
    if (!live || !at.inside)
        return;
    uint8_t *dst = place(at.which ? p.c.v : p.c.k, at) + at.lane4 * (D / 8);
    if (at.which) {
        // half words (2c, w) first, then (2c + 1, w)
        uint32_t h[GR];
#pragma unroll
        for (int w = 0; w < GR; w += 2) {
            h[w / 2] = __byte_perm(code[w], code[w + 1], 0x5410);
            h[GR / 2 + w / 2] = __byte_perm(code[w], code[w + 1], 0x7632);
        }
#pragma unroll
        for (int w = 0; w < GR; ++w)
            code[w] = h[w];
    }
    if constexpr (GR == 4)
        *reinterpret_cast<uint4 *>(dst) = make_uint4(code[0], code[1], code[2], code[3]);
    else
        *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
    if (at.lane4 == 0) {
        uint8_t *sd = place(at.which ? p.c.vs : p.c.ks, at);
        if constexpr (GR == 4)
            *reinterpret_cast<uint2 *>(sd) = make_uint2(scale[0], scale[1]);
        else
            *reinterpret_cast<uint32_t *>(sd) = scale[0];
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) get_rows_q4_kernel(const __grid_constant__ RowsQ4 p)
{
    constexpr int GR = D / 32;
    pdl_wait();
    pdl_trigger();
    Where at;
    if (!locate(p, &at))
        return;
    uint32_t code[GR], scale[GR / 2];
#pragma unroll
    for (int w = 0; w < GR; ++w)
        code[w] = 0x88888888u;
#pragma unroll
    for (int w = 0; w < GR / 2; ++w)
        scale[w] = 0u;
    if (at.inside) {
        const uint8_t *src = place(at.which ? p.c.v : p.c.k, at) + at.lane4 * (D / 8);
        const uint8_t *ss = place(at.which ? p.c.vs : p.c.ks, at);
        if constexpr (GR == 4) {
            const uint4 a = *reinterpret_cast<const uint4 *>(src);
            const uint2 b = *reinterpret_cast<const uint2 *>(ss);
            code[0] = a.x; code[1] = a.y; code[2] = a.z; code[3] = a.w;
            scale[0] = b.x; scale[1] = b.y;
        } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(src);
            code[0] = a.x; code[1] = a.y;
            scale[0] = *reinterpret_cast<const uint32_t *>(ss);
        }
    }
    if (at.which) {
        uint32_t h[GR];
#pragma unroll
        for (int w = 0; w < GR; w += 2) {
            h[w] = __byte_perm(code[w / 2], code[GR / 2 + w / 2], 0x5410);
            h[w + 1] = __byte_perm(code[w / 2], code[GR / 2 + w / 2], 0x7632);
        }
#pragma unroll
        for (int w = 0; w < GR; ++w)
            code[w] = h[w];
    }
    __nv_bfloat16 *dst = p.x[at.which] + at.t * p.ts[at.which] + at.head * D + 8 * at.lane4;
#pragma unroll
    for (int w = 0; w < GR; ++w) {
        // two elements a register, i and i + 4; every step is exact in bf16
        const uint32_t s2 = w & 1 ? __byte_perm(scale[w / 2], 0, 0x3232)
                                  : __byte_perm(scale[w / 2], 0, 0x1010);
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t n = sub136(nibbles(code[w], i));
            const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&n),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&s2));
            x[i] = *reinterpret_cast<const uint32_t *>(&y);
        }
        st_stream(dst + 32 * w,
                  make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                             __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632)));
    }
}

RowsQ4 pack_args(const CacheView &c, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                 const int64_t *rows, int64_t T, int64_t k_ts, int64_t v_ts, unsigned *status)
{
    RowsQ4 p = {};
    p.c = c;
    p.x[0] = const_cast<__nv_bfloat16 *>(k);
    p.x[1] = const_cast<__nv_bfloat16 *>(v);
    p.ts[0] = k_ts;
    p.ts[1] = v_ts;
    p.rows = rows;
    p.T = T;
    p.status = status;
    return p;
}

cudaError_t run(bool set, const RowsQ4 &p, cudaStream_t stream, LaunchRecord *rec)
{
    const int64_t threads = p.T * p.c.Hkv * 8;
    const int64_t grid = (threads + kThreads - 1) / kThreads;
    auto fn = set ? (p.c.D == 64 ? set_rows_q4_kernel<64> : set_rows_q4_kernel<128>)
                  : (p.c.D == 64 ? get_rows_q4_kernel<64> : get_rows_q4_kernel<128>);
    cudaError_t e = launch(fn, dim3((unsigned)grid), dim3(kThreads), 0, stream, 1, p);
    if (e == cudaSuccess && rec) {
        *rec = LaunchRecord();
        rec->kernel = set ? QKR_KERNEL_SET_ROWS_Q4 : QKR_KERNEL_GET_ROWS_Q4;
        rec->lanes_per_row = 4;
        rec->block = kThreads;
        rec->grid = grid;
        rec->launches = 1;
    }
    return e;
}

}  // namespace

cudaError_t launch_set_rows_q4(const CacheView &c, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                               const int64_t *rows, int64_t T, int64_t k_ts, int64_t v_ts,
                               unsigned *status, cudaStream_t stream, LaunchRecord *rec)
{
    return run(true, pack_args(c, k, v, rows, T, k_ts, v_ts, status), stream, rec);
}

cudaError_t launch_get_rows_q4(const CacheView &c, __nv_bfloat16 *k, __nv_bfloat16 *v,
                               const int64_t *rows, int64_t T, int64_t k_ts, int64_t v_ts,
                               unsigned *status, cudaStream_t stream, LaunchRecord *rec)
{
    return run(false, pack_args(c, k, v, rows, T, k_ts, v_ts, status), stream, rec);
}

}  // namespace qkr
