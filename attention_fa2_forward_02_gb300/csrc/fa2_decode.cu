// fa2_decode.cu - sizes and dispatch of the attention of one new token (fa2_decode.cuh), whose
// kernels are compiled per head size (fa2_decode_d32.cu, _d64.cu, _d128.cu).
#include "fa2_decode.cuh"

namespace fa2 {

size_t decode_workspace_bytes(int heads, int hkv, int d) {
    const bool one = heads / hkv <= 8;
    switch (pad_head_dim(d)) {
        case 32: return one ? workspace_for<32, 1>() : workspace_for<32, 2>();
        case 64: return one ? workspace_for<64, 1>() : workspace_for<64, 2>();
        default: return one ? workspace_for<128, 1>() : workspace_for<128, 2>();
    }
}

cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream) {
    switch (pad_head_dim(p.c.d)) {
        case 32: return launch_decode_d32(p, stream);
        case 64: return launch_decode_d64(p, stream);
        default: return launch_decode_d128(p, stream);
    }
}

}  // namespace fa2
