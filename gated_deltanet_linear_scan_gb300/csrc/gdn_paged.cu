// gdn_paged.cu -- tensor maps of the paged cache.
#include "gdn_paged.cuh"

namespace gdn {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library does not link against libcuda).
EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

CUtensorMapDataType map_type(int dtype) {
    return dtype == GDN_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
           : dtype == GDN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                              : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

gdn_status encode(CUtensorMap *map, const void *base, int dtype, int rank, const cuuint64_t *dims,
                  const cuuint64_t *strides, const cuuint32_t *box) {
    const EncodeTiled fn = encoder();
    if (fn == nullptr) return GDN_ERR_LAUNCH;
    const cuuint32_t unit[3] = {1, 1, 1};
    auto encode_once = [&] {
        return fn(map, map_type(dtype), static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims,
                  strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    if (encode_once() == CUDA_SUCCESS) return GDN_OK;
    // A driver call, it wants the device's context to be current, which in a host thread that has not
    // used the GPU yet it is not: the runtime makes it so where the thread's device is set.
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || cudaSetDevice(device) != cudaSuccess) return GDN_ERR_LAUNCH;
    return encode_once() == CUDA_SUCCESS ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

gdn_status encode_blocks_map(CUtensorMap *map, const void *base, int dtype, int cols, uint64_t rows,
                             uint64_t row_bytes, int box_rows, int box_blocks) {
    const int per = 128 / dtype_bytes(dtype);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(per), rows, static_cast<cuuint64_t>(cols / per)};
    const cuuint64_t strides[2] = {row_bytes, 128};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(per), static_cast<cuuint32_t>(box_rows),
                               static_cast<cuuint32_t>(box_blocks)};
    return encode(map, base, dtype, 3, dims, strides, box);
}

gdn_status encode_heads_map(CUtensorMap *map, const void *base, int dtype, int cols, int heads,
                            uint64_t tokens, uint64_t token_bytes, int box_heads, int box_tokens) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(heads),
                                tokens};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * dtype_bytes(dtype), token_bytes};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / dtype_bytes(dtype)),
                               static_cast<cuuint32_t>(box_heads),
                               static_cast<cuuint32_t>(box_tokens)};
    return encode(map, base, dtype, 3, dims, strides, box);
}

}  // namespace gdn
