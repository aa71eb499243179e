// fa2_selected_d64.cu - the kernels of fa2_decode.cuh over a block table for each key-value head, for head sizes 33 to 64.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 176 .. 191 of ensure_smem_limit
cudaError_t launch_selected_d64(const DecodeParams& p, cudaStream_t stream) { return launch_kind<64, true>(p, stream, 176); }

}  // namespace fa2
