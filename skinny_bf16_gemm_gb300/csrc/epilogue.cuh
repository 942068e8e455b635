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

// The activation of n values; one branch, not one a value. The GELUs by the complement,
// v erfc(-v / sqrt 2) / 2, and by v / (1 + exp(-2u)) = v (1 + tanh u) / 2: 1 + erf and 1 + tanh
// cancel for negative v (30 % off at -5, 0 from -5.5 on). Where the exponential overflows the
// value is under 1e-36 and comes out as -0. The approximate quotient is 2 ulp off (64 x 18432
// x 7168: 47.6 us, 50.3 with the IEEE one); erfcf costs 1 us more there than erff did.
template <int n>
__device__ __forceinline__ void activate(float (&v)[n], int activation) {
    switch (activation) {
        case kActRelu:
#pragma unroll
            for (int i = 0; i < n; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];  // NaN stays
            break;
        case kActSilu:
#pragma unroll
            for (int i = 0; i < n; ++i) v[i] = __fdiv_rn(v[i], 1.0f + expf(-v[i]));
            break;
        case kActGelu:
#pragma unroll
            for (int i = 0; i < n; ++i) v[i] = 0.5f * v[i] * erfcf(v[i] * -0.70710678118654752f);
            break;
        case kActGeluTanh:
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float u2 = 1.59576912160573071f * (v[i] + 0.044715f * v[i] * v[i] * v[i]);  // 2u
                v[i] = __fdividef(v[i], 1.0f + expf(-u2));
            }
            break;
        default: break;
    }
}

}  // namespace skinny
