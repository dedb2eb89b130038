// Packed-sequence attention forward (bf16), plans with a window.
#include "seq_fwd.cuh"

namespace sga {

template cudaError_t seq_fwd_bf16<true>(const SeqArgs &, int, cudaStream_t);

}  // namespace sga
