// fa2_decode_e2m1_d64.cu - the kernels of fa2_decode.cuh over 4-bit rows, for head size 64.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 128 .. 143 of ensure_smem_limit
cudaError_t launch_decode_e2m1_d64(const DecodeParams& p, cudaStream_t stream) { return launch_e2m1<64, false>(p, stream, 128); }

}  // namespace fa2
