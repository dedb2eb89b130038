// Packed-sequence attention backward (bf16), plans with a window.
#include "seq_bwd.cuh"

namespace sga {

template cudaError_t seq_bwd_bf16<true>(const SeqArgs &, int, cudaStream_t);

}  // namespace sga
