// fa2_selected_d128.cu - the kernels of fa2_decode.cuh over a block table for each key-value head, for head sizes 65 to 128.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 192 .. 207 of ensure_smem_limit
cudaError_t launch_selected_d128(const DecodeParams& p, cudaStream_t stream) { return launch_kind<128, true>(p, stream, 192); }

}  // namespace fa2
