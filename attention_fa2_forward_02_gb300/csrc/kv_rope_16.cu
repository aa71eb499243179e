// kv_rope_16.cu - the kernels of kv_rope.cuh into 16-bit rows.
#include "kv_rope.cuh"

namespace fa2 {

cudaError_t launch_rope_append_16(const RopeAppendParams& p, cudaStream_t stream) { return launch_form<kRows16>(p, stream); }

}  // namespace fa2
