// api_common.h -- argument checks, tensor-map encoding and small helpers that the extern "C"
// entry points share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "sfi.h"
#include "sfi_internal.h"

namespace sfi {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2-D bf16 view [rows][128] with 256-byte rows; box = 64 columns x box_rows rows, 128-byte
// swizzle (the canonical K-major / MN-major operand layout of the UMMA descriptors).
inline bool make_map(CUtensorMap *m, const void *base, uint64_t rows, uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn || rows == 0)
        return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kHeadDim), rows};
    const cuuint64_t strides[1] = {kHeadDim * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries of a packed chunk as [rows][heads][128]; a box is one kv head's G heads of
// box_rows / G rows (box_rows operand rows, by position, then head), 64 columns, 128-byte
// swizzle.
inline bool make_chunk_map(CUtensorMap *m, const void *base, uint64_t rows, uint32_t heads, uint32_t group,
                           uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn || rows == 0)
        return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), heads, rows};
    const cuuint64_t strides[2] = {kHeadDim * 2, static_cast<cuuint64_t>(heads) * kHeadDim * 2};
    const cuuint32_t box[3] = {64, group, box_rows / group};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline sfi_status check_kv(const sfi_kv_cache *kv)
{
    if (!kv || !kv->k || !kv->v || !kv->seq_len || !kv->err)
        return SFI_ERR_INVALID_ARG;
    if (kv->n_layers < 1 || kv->batch < 1 || kv->n_kv_heads < 1 || kv->n_q_heads < 1)
        return SFI_ERR_INVALID_ARG;
    if (kv->head_dim != kHeadDim || kv->batch > kMaxBatch)
        return SFI_ERR_UNSUPPORTED;
    if (kv->n_q_heads % kv->n_kv_heads != 0)
        return SFI_ERR_INVALID_ARG;
    const int g = kv->n_q_heads / kv->n_kv_heads;
    if (g != 1 && g != 2 && g != 4 && g != 8)
        return SFI_ERR_UNSUPPORTED;
    if (!aligned16(kv->k) || !aligned16(kv->v))
        return SFI_ERR_INVALID_ARG;
    if (kv->max_len < 0 || kv->capacity < 1)
        return SFI_ERR_INVALID_ARG;
    if (kv->page_size != 0) {
        if (kv->page_size != 16)
            return SFI_ERR_UNSUPPORTED;
        if (!kv->page_table || kv->n_pages < 1 || kv->max_pages_per_seq < 1 ||
            kv->capacity != kv->max_pages_per_seq * kv->page_size)
            return SFI_ERR_INVALID_ARG;
    }
    if (kv->max_len > kv->capacity)
        return SFI_ERR_CAPACITY;
    const long long units = 1LL * kv->n_layers * kv->batch * kv->n_kv_heads;
    const long long rows = kv->page_size ? 1LL * kv->n_layers * kv->n_pages * kv->n_kv_heads * 16
                                         : units * kv->capacity;
    if (units > 65535 || rows >= (1LL << 31))
        return SFI_ERR_UNSUPPORTED;
    return SFI_OK;
}

inline sfi_status check_budget(const sfi_budget *bd)
{
    if (!bd || bd->n_sink < 0 || bd->n_window < 1 || bd->n_select < 0 || bd->prior_tau < 1)
        return SFI_ERR_INVALID_ARG;
    if ((bd->prior_tau & (bd->prior_tau - 1)) != 0 || !(bd->lambda >= 0.0 && bd->lambda <= 1.0))
        return SFI_ERR_INVALID_ARG;
    if (bd->n_sink + bd->n_select < 1)
        return SFI_ERR_INVALID_ARG;
    return SFI_OK;
}

inline int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }

inline sfi_status launch_status(cudaError_t e) { return e == cudaSuccess ? SFI_OK : SFI_ERR_CUDA; }

inline uint64_t cache_rows(const sfi_kv_cache *kv)
{
    if (kv->page_size)
        return static_cast<uint64_t>(kv->n_layers) * kv->n_pages * kv->n_kv_heads * kv->page_size;
    return static_cast<uint64_t>(kv->n_layers) * kv->batch * kv->n_kv_heads * kv->capacity;
}

}  // namespace sfi
