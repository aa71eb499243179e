// fa2_decode.cu - sizes and dispatch of the attention of one new token (fa2_decode.cuh), whose
// kernels are compiled per head size (fa2_decode_d32.cu, _d64.cu, _d128.cu).
#include "fa2_decode.cuh"

namespace fa2 {

size_t decode_workspace_bytes(int heads, int hkv, int d, bool e2m1) {
    const bool one = heads / hkv <= 8;
    switch (pad_head_dim(d)) {
        case 32: return one ? workspace_for<32, 1>(e2m1) : workspace_for<32, 2>(e2m1);
        case 64: return one ? workspace_for<64, 1>(e2m1) : workspace_for<64, 2>(e2m1);
        default: return one ? workspace_for<128, 1>(e2m1) : workspace_for<128, 2>(e2m1);
    }
}

cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream) {
    if (p.c.form == kRowsE2m1) {
        switch (pad_head_dim(p.c.d)) {
            case 32: return p.per_head ? launch_selected_e2m1_d32(p, stream) : launch_decode_e2m1_d32(p, stream);
            case 64: return p.per_head ? launch_selected_e2m1_d64(p, stream) : launch_decode_e2m1_d64(p, stream);
            default: return p.per_head ? launch_selected_e2m1_d128(p, stream) : launch_decode_e2m1_d128(p, stream);
        }
    }
    switch (pad_head_dim(p.c.d)) {
        case 32: return p.per_head ? launch_selected_d32(p, stream) : launch_decode_d32(p, stream);
        case 64: return p.per_head ? launch_selected_d64(p, stream) : launch_decode_d64(p, stream);
        default: return p.per_head ? launch_selected_d128(p, stream) : launch_decode_d128(p, stream);
    }
}

}  // namespace fa2
