// decode_attention_shared_prefix_bf16 in one launch, for prefixes that are little work
// (decode_attention_kernel.cuh), a file of its own so that the forms compile at once.
#include "decode_attention_kernel.cuh"

namespace skinny {

cudaError_t launch_decode_attention_joined(const SharedAttentionArgs &a, int head_dim, int num_sms, int device,
                                           cudaStream_t stream, bool pdl) {
    return launch_any_dim<kJoined>(a, head_dim, num_sms, device, stream, pdl);
}

cudaError_t attention_joined_error_word(int **word) { return error_word(word); }

}  // namespace skinny
