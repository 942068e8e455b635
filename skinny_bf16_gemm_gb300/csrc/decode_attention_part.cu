// The rows' own tokens of decode_attention_shared_prefix_bf16 (decode_attention_kernel.cuh), a
// file of its own so that the forms compile at once.
#include "decode_attention_kernel.cuh"

namespace skinny {

cudaError_t launch_decode_attention_part(const SharedAttentionArgs &a, int head_dim, int num_sms, int device,
                                         cudaStream_t stream) {
    // Behind the prefix's kernel, which waits for what was before both.
    return launch_any_dim<kPart>(a, head_dim, num_sms, device, stream, true);
}

cudaError_t attention_part_error_word(int **word) { return error_word(word); }

}  // namespace skinny
