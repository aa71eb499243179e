// fa2_selected_e2m1_d64.cu - the kernels of fa2_decode.cuh over 4-bit rows and a block table for each key-value head, for head size 64.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 256 .. 271 of ensure_smem_limit
cudaError_t launch_selected_e2m1_d64(const DecodeParams& p, cudaStream_t stream) { return launch_e2m1<64, true>(p, stream, 256); }

}  // namespace fa2
