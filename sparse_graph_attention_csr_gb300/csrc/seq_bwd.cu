// Packed-sequence attention backward (bf16), plans without a window.
#include "seq_bwd.cuh"

namespace sga {

template cudaError_t seq_bwd_bf16<false>(const SeqArgs &, int, cudaStream_t);

}  // namespace sga
