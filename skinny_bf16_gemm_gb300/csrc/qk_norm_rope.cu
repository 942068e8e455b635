// Per-head RMSNorm of queries and keys with the position rotation in the same pass,
// and the append of keys and values to a paged cache, on GB300 (sm_103a).
//
// Per query or key head x[0..D) of a row at position p, FP32 throughout:
//   y = (x * rsqrt(sum(x^2) / D + eps)) * gamma
//   (a, b) -> (a cos - b sin, b cos + a sin) for the rot/2 pairs of the first rot
//   values ((i, i + rot/2), or (2i, 2i + 1) interleaved), angles from the table row p;
// one BF16 rounding at the end. Value heads are copied. Bound by HBM for many rows
// (each head read once, written once) and by latency for a few.
//
// Layout: a group of L lanes (8, 16 or 32: the smallest that covers D / 8) holds a
// head, 16 bytes to a lane, so the norm is a butterfly within the group and the
// half-split partner one shuffle away; a block has one row's heads, U to a group, so
// the table row is read once into registers for them. U = 4 keeps four loads in flight
// per lane for long inputs, U = 1 spreads few rows over the most threads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"

namespace skinny {
namespace {

constexpr int kMaxThreads = 512;
__device__ int g_rope_err;  // nonzero: a position or slot was out of range

__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = static_cast<uint32_t>(__bfloat16_as_ushort(b.x)) |
               (static_cast<uint32_t>(__bfloat16_as_ushort(b.y)) << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int L, int U>
__global__ void __launch_bounds__(kMaxThreads, 2) qk_norm_rope_kernel(const RopeArgs a) {
    const int groups = blockDim.x / L;
    const int lane = threadIdx.x % L;
    const int group = threadIdx.x / L;
    const int row = blockIdx.x;
    const bool active = lane * 8 < a.head_dim;
    const int heads = a.q_heads + 2 * a.kv_heads;
    const int head0 = blockIdx.y * (groups * U) + group;

    // The gammas are weights: read before waiting for the previous kernel.
    uint4 gq = make_uint4(0, 0, 0, 0), gk = gq;
    if (active && a.q_gamma != nullptr) gq = __ldg(reinterpret_cast<const uint4 *>(a.q_gamma) + lane);
    if (active && a.k_gamma != nullptr) gk = __ldg(reinterpret_cast<const uint4 *>(a.k_gamma) + lane);
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();  // rows, positions and slots may be the previous kernel's output

    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = head0 + u * groups;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (active && h < heads)
            raw[u] = __ldcs(reinterpret_cast<const uint4 *>(a.qkv + row * a.qkv_stride +
                                                            static_cast<long long>(h) * a.head_dim) + lane);
    }

    // The table row: lane's 8 values rotate with 8 angles (half-split: those of the
    // pair index i mod rot/2) or 4 (interleaved).
    const int half = a.rot_dim / 2;
    const bool turns = lane * 8 < a.rot_dim;
    float c[8], s[8];
    bool good = true;
    if (a.rot_dim > 0) {
        const int p = __ldcg(a.positions + row);
        good = p >= 0 && p < a.max_pos;
        if (turns && good) {
            const float *t = a.rope + static_cast<long long>(p) * a.rot_dim;
            if (a.interleaved) {
                const float4 c4 = *reinterpret_cast<const float4 *>(t + lane * 4);
                const float4 s4 = *reinterpret_cast<const float4 *>(t + half + lane * 4);
                c[0] = c4.x; c[1] = c4.y; c[2] = c4.z; c[3] = c4.w;
                s[0] = s4.x; s[1] = s4.y; s[2] = s4.z; s[3] = s4.w;
            } else {
                const int i = lane * 8 < half ? lane * 8 : lane * 8 - half;
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const float4 c4 = *reinterpret_cast<const float4 *>(t + i + j);
                    const float4 s4 = *reinterpret_cast<const float4 *>(t + half + i + j);
                    c[j] = c4.x; c[j + 1] = c4.y; c[j + 2] = c4.z; c[j + 3] = c4.w;
                    s[j] = s4.x; s[j + 1] = s4.y; s[j + 2] = s4.z; s[j + 3] = s4.w;
                }
            }
        }
    }
    long long cache_off = -1;  // this row's element offset in the pools, -1: not stored
    if (a.k_cache != nullptr) {
        const long long slot = __ldcg(a.slots + row);
        if (slot >= static_cast<long long>(a.num_pages) * a.page_size) {
            good = false;
        } else if (slot >= 0) {
            const long long page = slot / a.page_size;
            cache_off = page * a.page_stride + (slot - page * a.page_size) * a.token_stride;
        }
    }
    if (!good) {
        // Out of range: nothing of the row is written, the host can read the word.
        if (threadIdx.x == 0) atomicOr(&g_rope_err, 1);
        return;
    }

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = head0 + u * groups;
        if (h - group >= heads) break;  // past the last head for every group of the block
        const bool is_v = h >= a.q_heads + a.kv_heads, is_q = h < a.q_heads;
        uint4 w = raw[u];
        float y[8];
        unpack(w, y);
        // Every lane of the warp takes part in the shuffles; results of value heads
        // and of heads past the end are dropped.
        if (is_q ? a.q_gamma != nullptr : a.k_gamma != nullptr) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
            float g[8];
            unpack(is_q ? gq : gk, g);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1)
                ss += __shfl_xor_sync(L == 32 ? 0xFFFFFFFFu : ((1u << (L & 31)) - 1u) << (threadIdx.x % 32 / L * L), ss, o);
            const float rstd = rsqrtf(__fdiv_rn(ss, static_cast<float>(a.head_dim)) + a.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = y[j] * rstd * g[j];
        }
        if (a.rot_dim > 0) {
            if (a.interleaved) {
                if (turns) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = y[2 * j], q = y[2 * j + 1];
                        y[2 * j] = p * c[j] - q * s[j];
                        y[2 * j + 1] = q * c[j] + p * s[j];
                    }
                }
            } else {
                const int hl = half / 8;  // lanes of half the rotated part
                const int partner = lane < hl ? lane + hl : lane - hl;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float o = __shfl_sync(0xFFFFFFFFu, y[j], turns ? partner : lane, L);
                    if (turns) y[j] = lane < hl ? y[j] * c[j] - o * s[j] : y[j] * c[j] + o * s[j];
                }
            }
        }
        if (!active || h >= heads) continue;
        if (!is_v) w = pack(y);
        if (is_q) {
            reinterpret_cast<uint4 *>(a.q_out + row * a.q_stride + static_cast<long long>(h) * a.head_dim)[lane] = w;
            continue;
        }
        const int kh = h - a.q_heads - (is_v ? a.kv_heads : 0);
        if (!is_v && a.k_out != nullptr)
            reinterpret_cast<uint4 *>(a.k_out + row * a.k_stride + static_cast<long long>(kh) * a.head_dim)[lane] = w;
        if (cache_off >= 0)
            reinterpret_cast<uint4 *>((is_v ? a.v_cache : a.k_cache) + cache_off + kh * a.head_stride)[lane] = w;
    }
}

template <int L, int U>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream, bool pdl) {
    // Blocks of a row just large enough for their share of its heads.
    const int heads = a.q_heads + 2 * a.kv_heads, most = kMaxThreads / L * U;
    const int blocks = (heads + most - 1) / most, share = (heads + blocks - 1) / blocks;
    const int threads = ((share + U - 1) / U * L + 31) / 32 * 32, per_block = threads / L * U;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.rows, (heads + per_block - 1) / per_block, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<L, U>, a);
}

template <int L>
cudaError_t launch_lanes(const RopeArgs &a, cudaStream_t stream, bool pdl) {
    // Few heads in all: one per group, so that they spread over the SMs.
    const long long heads = static_cast<long long>(a.rows) * (a.q_heads + 2 * a.kv_heads);
    if (heads * L < 152ll * 2048) return launch<L, 1>(a, stream, pdl);
    return launch<L, 4>(a, stream, pdl);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs &a, cudaStream_t stream, bool pdl) {
    if (a.head_dim <= 64) return launch_lanes<8>(a, stream, pdl);
    if (a.head_dim <= 128) return launch_lanes<16>(a, stream, pdl);
    return launch_lanes<32>(a, stream, pdl);
}

cudaError_t rope_error_word(int *value, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_rope_err, sizeof(int));
    if (e != cudaSuccess || !clear || *value == 0) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_rope_err, &zero, sizeof(int));
}

}  // namespace skinny
