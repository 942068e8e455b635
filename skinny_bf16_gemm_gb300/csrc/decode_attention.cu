// decode_attention_bf16 (decode_attention_kernel.cuh).
#include "decode_attention_kernel.cuh"

namespace skinny {

cudaError_t launch_decode_attention(const AttentionArgs &a, int head_dim, int num_sms, int device,
                                    cudaStream_t stream, bool pdl) {
    return launch_any_dim<kWhole>(a, head_dim, num_sms, device, stream, pdl);
}

cudaError_t attention_error_word(int **word) { return error_word(word); }

}  // namespace skinny
