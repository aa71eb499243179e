// fa2_decode_e2m1_d32.cu - the kernels of fa2_decode.cuh over 4-bit rows, for head size 32.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 112 .. 127 of ensure_smem_limit
cudaError_t launch_decode_e2m1_d32(const DecodeParams& p, cudaStream_t stream) { return launch_e2m1<32, false>(p, stream, 112); }

}  // namespace fa2
