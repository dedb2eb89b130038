// Packed-sequence attention forward (bf16), plans without a window; and the tensor
// maps of both passes.
#include "seq_fwd.cuh"

namespace sga {

cudaError_t seq_tensor_map(CUtensorMap *m, const void *base, int64_t rows, int heads, int D, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode;
    if (cudaError_t e = tmap_encoder(encode); e != cudaSuccess) return e;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, estr[3] = {1, 1, 1};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template cudaError_t seq_fwd_bf16<false>(const SeqArgs &, int, cudaStream_t);

}  // namespace sga
