// kv_rope_e2m1.cu - the kernels of kv_rope.cuh into 4-bit rows.
#include "kv_rope.cuh"

namespace fa2 {

cudaError_t launch_rope_append_e2m1(const RopeAppendParams& p, cudaStream_t stream) { return launch_form<kRowsE2m1>(p, stream); }

}  // namespace fa2
