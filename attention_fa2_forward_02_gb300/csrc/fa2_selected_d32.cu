// fa2_selected_d32.cu - the kernels of fa2_decode.cuh over a block table for each key-value head, for head sizes up to 32.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 160 .. 175 of ensure_smem_limit
cudaError_t launch_selected_d32(const DecodeParams& p, cudaStream_t stream) { return launch_kind<32, true>(p, stream, 160); }

}  // namespace fa2
