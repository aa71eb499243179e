// fa2_decode_e2m1_d128.cu - the kernels of fa2_decode.cuh over 4-bit rows, for head sizes 96 and 128.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 144 .. 159 of ensure_smem_limit
cudaError_t launch_decode_e2m1_d128(const DecodeParams& p, cudaStream_t stream) { return launch_e2m1<128, false>(p, stream, 144); }

}  // namespace fa2
