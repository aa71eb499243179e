// fa2_decode_d64.cu - the kernels of fa2_decode.cuh for head sizes 33 to 64.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 80 .. 95 of ensure_smem_limit (the attention kernels take 0 .. 61)
cudaError_t launch_decode_d64(const DecodeParams& p, cudaStream_t stream) { return launch_kind<64>(p, stream, 80); }

}  // namespace fa2
