// kv_rope_e4m3.cu - the kernels of kv_rope.cuh into 8-bit rows.
#include "kv_rope.cuh"

namespace fa2 {

cudaError_t launch_rope_append_e4m3(const RopeAppendParams& p, cudaStream_t stream) { return launch_form<kRowsE4m3>(p, stream); }

}  // namespace fa2
