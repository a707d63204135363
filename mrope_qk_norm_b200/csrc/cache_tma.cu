// cache_tma.cu -- tensor maps over the rows of a cache, encoded on the host by
// the driver for each call.

#include "cache_tma.cuh"

#include <atomic>

namespace qkr {
namespace {

// The driver's tensor-map encoder, without linking the driver library.
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encoder(EncodeFn *fn)
{
    static std::atomic<EncodeFn> found{nullptr};   // the same address for every caller
    EncodeFn have = found.load(std::memory_order_relaxed);
    if (!have) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult res;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                         cudaEnableDefault, &res);
        if (e != cudaSuccess)
            return e;
        if (res != cudaDriverEntryPointSuccess || !f)
            return cudaErrorNotSupported;
        have = reinterpret_cast<EncodeFn>(f);
        found.store(have, std::memory_order_relaxed);
    }
    *fn = have;
    return cudaSuccess;
}

cudaError_t encode(EncodeFn fn, const CacheView &c, const CachePlane &pl, bool q4, int box,
                   PlaneMap *out)
{
    int page_axis;
    // axes by stride; the stride of an axis of one is free, so it goes last
    struct Axis {
        int64_t stride, extent;
        int box, *at;
    } ax[3] = {{pl.rs, c.page_size, box, &out->row_axis},
               {pl.hs, c.Hkv, 1, &out->head_axis},
               {pl.ps, c.n_pages, 1, &page_axis}};
    for (Axis &a : ax)
        if (a.extent == 1)
            a.stride = (int64_t)1 << 39;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (ax[j].stride > ax[j + 1].stride) {
                const Axis t = ax[j];
                ax[j] = ax[j + 1];
                ax[j + 1] = t;
            }
    cuuint64_t dims[4] = {(cuuint64_t)(q4 ? c.D / 2 : c.D), 0, 0, 0}, strides[3];
    cuuint32_t boxes[4] = {(cuuint32_t)(q4 ? c.D / 2 : 64), 0, 0, 0}, steps[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        dims[i + 1] = (cuuint64_t)ax[i].extent;
        strides[i] = (cuuint64_t)ax[i].stride;
        boxes[i + 1] = (cuuint32_t)ax[i].box;
        *ax[i].at = i + 1;
    }
    out->box = box;
    const CUresult r =
        fn(&out->m, q4 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pl.base,
           dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
           !q4 ? CU_TENSOR_MAP_SWIZZLE_128B
               : (c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE),
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t cache_maps(const CacheView &c, bool q4, int keys, CacheMaps *maps)
{
    EncodeFn fn;
    cudaError_t e = encoder(&fn);
    int box = keys;
    while (c.page_size % box)
        box /= 2;
    if (e == cudaSuccess)
        e = encode(fn, c, c.k, q4, box, &maps->k);
    if (e == cudaSuccess)
        e = encode(fn, c, c.v, q4, box, &maps->v);
    return e;
}

}  // namespace qkr
