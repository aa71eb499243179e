// fa2_decode_d32.cu - the kernels of fa2_decode.cuh for head sizes up to 32.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 64 .. 79 of ensure_smem_limit (the attention kernels take 0 .. 61)
cudaError_t launch_decode_d32(const DecodeParams& p, cudaStream_t stream) { return launch_kind<32>(p, stream, 64); }

}  // namespace fa2
