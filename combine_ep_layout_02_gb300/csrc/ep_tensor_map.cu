// ep_tensor_map.cu -- host side: TMA descriptors.  They are encoded for every
// call and travel as kernel parameters; nothing is kept between calls.
#include "ep_tcgen05.cuh"

namespace ep {
namespace {

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once per process.
cudaError_t encoder(Encode* out) {
    static std::atomic<void*> entry{nullptr};
    void* fn = entry.load(std::memory_order_acquire);
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        const cudaError_t err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                                 cudaEnableDefault, &found);
        if (err != cudaSuccess) return err;
        if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        entry.store(fn, std::memory_order_release);
    }
    *out = reinterpret_cast<Encode>(fn);
    return cudaSuccess;
}

cudaError_t encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box,
                   CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8) {
    Encode fn;
    const cudaError_t err = encoder(&fn);
    if (err != cudaSuccess) return err;
    const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
    const CUresult r = fn(map, type, (cuuint32_t)rank, const_cast<void*>(base),
                          dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t byte_matrix_map(CUtensorMap* map, const void* base, int64_t rows, int64_t width,
                            int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)width};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    return encode(map, base, 2, dims, strides, box);
}

cudaError_t byte_blocks_map(CUtensorMap* map, const void* base, int64_t rows, int64_t width,
                            int box_rows, int blocks) {
    const cuuint64_t dims[3] = {128, (cuuint64_t)rows, (cuuint64_t)(width / 128)};
    const cuuint64_t strides[2] = {(cuuint64_t)width, 128};
    const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, (cuuint32_t)blocks};
    return encode(map, base, 3, dims, strides, box);
}

cudaError_t typed_map(CUtensorMap* map, int type, const void* base, int rank, const uint64_t* dims,
                      const uint64_t* strides, const uint32_t* box) {
    cuuint64_t d[5], s[4];
    cuuint32_t b[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i > 0) s[i - 1] = strides[i - 1];
    }
    return encode(map, base, rank, d, s, b,
                  type == EP_TYPE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

}  // namespace ep
