// fa2_selected_e2m1_d32.cu - the kernels of fa2_decode.cuh over 4-bit rows and a block table for each key-value head, for head size 32.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 240 .. 255 of ensure_smem_limit
cudaError_t launch_selected_e2m1_d32(const DecodeParams& p, cudaStream_t stream) { return launch_e2m1<32, true>(p, stream, 240); }

}  // namespace fa2
