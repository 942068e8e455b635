// The decode GEMM's optional epilogue: out = BF16(act(v + bias[n]) + residual[m][n]),
// v the FP32 sum over K. Every step is FP32 and the result is rounded once; a
// missing bias or residual is skipped, not added as zero, so that a call with
// neither and no activation gives decode_gemm_bf16's bits (-0 included).
#pragma once

#include <cstdint>

namespace skinny {

// Activation codes (skinny_activation of the C ABI).
enum Activation : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

struct Epilogue {
    const uint16_t *bias;      // [N] BF16 or nullptr
    const uint16_t *residual;  // [M, N] BF16 or nullptr; may be out itself
    int activation;
};

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

__device__ __forceinline__ float activate(float v, int activation) {
    switch (activation) {
        case kActRelu: return v < 0.0f ? 0.0f : v;  // NaN stays
        case kActSilu: return __fdiv_rn(v, 1.0f + expf(-v));
        case kActGelu: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
        case kActGeluTanh:
            return 0.5f * v * (1.0f + tanhf(0.79788456080286536f * (v + 0.044715f * v * v * v)));
        default: return v;
    }
}

}  // namespace skinny
