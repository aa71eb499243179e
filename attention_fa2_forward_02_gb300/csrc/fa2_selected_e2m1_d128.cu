// fa2_selected_e2m1_d128.cu - the kernels of fa2_decode.cuh over 4-bit rows and a block table for each key-value head, for head sizes 96 and 128.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 272 .. 287 of ensure_smem_limit
cudaError_t launch_selected_e2m1_d128(const DecodeParams& p, cudaStream_t stream) { return launch_e2m1<128, true>(p, stream, 272); }

}  // namespace fa2
