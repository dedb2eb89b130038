// Packed-sequence attention in fp32, plans without a window.
#include "seq_simt.cuh"

namespace sga {

template cudaError_t seq_fwd_f32<false>(const SeqArgs &, int, cudaStream_t);
template cudaError_t seq_bwd_f32<false>(const SeqArgs &, int, cudaStream_t);

}  // namespace sga
