// fa2_decode_d128.cu - the kernels of fa2_decode.cuh for head sizes 65 to 128.
#include "fa2_decode.cuh"

namespace fa2 {

// slots 96 .. 111 of ensure_smem_limit (the attention kernels take 0 .. 61)
cudaError_t launch_decode_d128(const DecodeParams& p, cudaStream_t stream) { return launch_kind<128>(p, stream, 96); }

}  // namespace fa2
