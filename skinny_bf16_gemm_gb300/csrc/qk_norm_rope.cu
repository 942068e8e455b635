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
// head, 8 values to a lane, so the norm is a butterfly within the group. Where heads are
// rotated by halves (HALVES) a lane has four values and their four partners, in two 8-byte
// pieces, so the rotation stays within the lane and needs 4 cosines and 4 sines; else
// 16 bytes side by side. A group does U heads of one kind (query, key or value), so its
// gamma stays in registers, and goes through the rows with the next row's heads and angles,
// and the position after that, on their way: blocks that did one row each waited out
// position, table and heads one after another, and more units a thread or more threads
// an SM spill. The arithmetic is on pairs (f32x2): heads of all kinds in one group, with
// scalar arithmetic, took 200 instructions a head and warp and were bound by them.
// U = 4 keeps the loads of four heads in flight, U = 1 spreads few rows over the most
// threads. Measured on GB300, 8191 rows of 56 + 2 x 8 heads of 128: 57 us, 5.3 TB/s
// (one row a block: 87 us; kinds mixed, scalar: 88 us; U = 2: 69 us; 768 threads an SM:
// 82 us); 64 rows 3.5 us and one row of 9 heads 2.2 us in a graph.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace skinny {
namespace {

constexpr int kMaxThreads = 128;  // of a block
constexpr int kResident = 512;    // of an SM: up to 128 registers each
__device__ int g_rope_err;  // nonzero: a position or slot was out of range

// Two FP32 values in a register pair; multiply, multiply-add and add round each.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float a, float b) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ float2 floats_of(Pair p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Pair unpack(uint32_t w) {  // two BF16 values
    return pair_of(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack(Pair p) {
    const float2 f = floats_of(p);
    const __nv_bfloat162 x = __floats2bfloat162_rn(f.x, f.y);
    return static_cast<uint32_t>(__bfloat16_as_ushort(x.x)) | (static_cast<uint32_t>(__bfloat16_as_ushort(x.y)) << 16);
}

template <int L, int U, bool HALVES>
__global__ void __launch_bounds__(kMaxThreads, kResident / kMaxThreads) qk_norm_rope_kernel(const RopeArgs a) {
    const int lane = threadIdx.x % L;
    const int group = blockIdx.y * (blockDim.x / L) + threadIdx.x / L;
    // This lane's two pieces of four values.
    const int half = a.rot_dim / 2;
    const bool turns = lane * 8 < a.rot_dim;
    const int at0 = HALVES && turns ? lane * 4 : lane * 8, at1 = HALVES && turns ? at0 + half : at0 + 4;
    auto load = [&](const uint16_t *from) -> uint4 {
        if constexpr (HALVES) {
            const uint2 x = __ldcs(reinterpret_cast<const uint2 *>(from + at0));
            const uint2 y = __ldcs(reinterpret_cast<const uint2 *>(from + at1));
            return make_uint4(x.x, x.y, y.x, y.y);
        } else {
            return __ldcs(reinterpret_cast<const uint4 *>(from + at0));
        }
    };

    // This group's heads: [first, first + count) of one kind, the same for every row. A
    // group past the last has none (and goes along for the warp's sake).
    enum Kind : int { kQuery, kKey, kValue };
    const int q_groups = (a.q_heads + U - 1) / U, kv_groups = (a.kv_heads + U - 1) / U;
    const int kind = group < q_groups ? kQuery : group < q_groups + kv_groups ? kKey : kValue;
    const int first = (group - (kind == kQuery ? 0 : q_groups + (kind == kKey ? 0 : kv_groups))) * U;
    const int count = max(0, min(U, (kind == kQuery ? a.q_heads : a.kv_heads) - first));
    const bool active = lane * 8 < a.head_dim && count > 0;
    const uint16_t *from = a.qkv + (first + (kind == kQuery ? 0 : a.q_heads + (kind == kKey ? 0 : a.kv_heads))) * a.head_dim;
    // The gammas are weights: read before waiting for the previous kernel.
    const uint16_t *gamma = kind == kQuery ? a.q_gamma : kind == kKey ? a.k_gamma : nullptr;
    Pair g[4] = {};
    if (active && gamma != nullptr) {
        const uint4 w = load(gamma);
        g[0] = unpack(w.x);
        g[1] = unpack(w.y);
        g[2] = unpack(w.z);
        g[3] = unpack(w.w);
    }
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();  // rows, positions and slots may be the previous kernel's output

    struct Where {
        int position;
        long long slot;
    };
    auto where = [&](int row) -> Where {
        Where w = {0, -1};
        if (row < a.rows) {
            if (a.rot_dim > 0) w.position = __ldcg(a.positions + row);
            if (a.k_cache != nullptr) w.slot = __ldcg(a.slots + row);
        }
        return w;
    };
    auto in_table = [&](int p) { return a.rot_dim == 0 || (p >= 0 && p < a.max_pos); };
    uint4 next[U] = {};  // stays zero in lanes past the head
    float4 next_c = {}, next_s = {};  // the table row's angles of this lane's four pairs
    auto fetch = [&](int row, int p) {
        if (row >= a.rows || !active) return;
        const uint16_t *at = from + row * a.qkv_stride;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < count) next[u] = load(at + u * a.head_dim);
        if (turns && kind != kValue && in_table(p)) {
            const float *t = a.rope + static_cast<long long>(p) * a.rot_dim + lane * 4;
            next_c = *reinterpret_cast<const float4 *>(t);
            next_s = *reinterpret_cast<const float4 *>(t + half);
        }
    };
    const unsigned mask = L == 32 ? 0xFFFFFFFFu : ((1u << (L & 31)) - 1u) << (threadIdx.x % 32 / L * L);
    int row = blockIdx.x;
    const int step = gridDim.x;
    Where here = where(row), after = where(row + step);
    fetch(row, here.position);
    for (; row < a.rows; row += step) {
        uint4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = next[u];
        const Pair c[2] = {pair_of(next_c.x, next_c.y), pair_of(next_c.z, next_c.w)};
        const Pair s[2] = {pair_of(next_s.x, next_s.y), pair_of(next_s.z, next_s.w)};
        const Pair minus_s[2] = {pair_of(-next_s.x, -next_s.y), pair_of(-next_s.z, -next_s.w)};
        const Where at = here;
        fetch(row + step, after.position);
        here = after;
        after = where(row + 2 * step);

        if (!in_table(at.position) || at.slot >= a.num_slots) {
            // Out of range: nothing of the row is written, the host can read the word.
            if (threadIdx.x == 0) atomicOr(&g_rope_err, 1);
            continue;
        }
        if (kind != kValue) {
            float rstd[U];
            if (gamma != nullptr) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    Pair ss = mul(unpack(w[u].x), unpack(w[u].x));
                    ss = fma(unpack(w[u].y), unpack(w[u].y), ss);
                    ss = fma(unpack(w[u].z), unpack(w[u].z), ss);
                    ss = fma(unpack(w[u].w), unpack(w[u].w), ss);
                    const float2 f = floats_of(ss);
                    rstd[u] = f.x + f.y;
                }
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int u = 0; u < U; ++u) rstd[u] += __shfl_xor_sync(mask, rstd[u], o);
#pragma unroll
                for (int u = 0; u < U; ++u) rstd[u] = rsqrtf(fmaf(rstd[u], a.inv_dim, a.eps));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                Pair y[4] = {unpack(w[u].x), unpack(w[u].y), unpack(w[u].z), unpack(w[u].w)};
                if (gamma != nullptr) {
                    const Pair r = pair_of(rstd[u], rstd[u]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = mul(mul(y[j], r), g[j]);
                }
                if (turns) {
                    if constexpr (HALVES) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const Pair x = y[j], z = y[j + 2];
                            y[j] = fma(x, c[j], mul(z, minus_s[j]));
                            y[j + 2] = fma(z, c[j], mul(x, s[j]));
                        }
                    } else {
                        // Neighbours: sort into firsts and seconds, turn, sort back.
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float2 p = floats_of(y[2 * j]), q = floats_of(y[2 * j + 1]);
                            const Pair x = pair_of(p.x, q.x), z = pair_of(p.y, q.y);
                            const float2 n = floats_of(fma(x, c[j], mul(z, minus_s[j])));
                            const float2 m = floats_of(fma(z, c[j], mul(x, s[j])));
                            y[2 * j] = pair_of(n.x, m.x);
                            y[2 * j + 1] = pair_of(n.y, m.y);
                        }
                    }
                }
                w[u] = make_uint4(pack(y[0]), pack(y[1]), pack(y[2]), pack(y[3]));
            }
        }
        if (!active) continue;
        auto store = [&](uint16_t *to, long long stride) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u >= count) break;
                if constexpr (HALVES) {
                    *reinterpret_cast<uint2 *>(to + at0) = make_uint2(w[u].x, w[u].y);
                    *reinterpret_cast<uint2 *>(to + at1) = make_uint2(w[u].z, w[u].w);
                } else {
                    *reinterpret_cast<uint4 *>(to + at0) = w[u];
                }
                to += stride;
            }
        };
        if (kind == kQuery) {
            store(a.q_out + row * a.q_stride + first * a.head_dim, a.head_dim);
            continue;
        }
        if (kind == kKey && a.k_out != nullptr) store(a.k_out + row * a.k_stride + first * a.head_dim, a.head_dim);
        if (at.slot >= 0) {
            const long long page = a.page_shift >= 0 ? at.slot >> a.page_shift : at.slot / a.page_size;
            store((kind == kKey ? a.k_cache : a.v_cache) + page * a.page_stride +
                      (at.slot - page * a.page_size) * a.token_stride + first * a.head_stride,
                  a.head_stride);
        }
    }
}

template <int L, int U, bool HALVES>
cudaError_t launch(const RopeArgs &a, int num_sms, cudaStream_t stream, bool pdl) {
    // A row's groups in blocks of equal size, and as many blocks as stay on the GPU at once.
    const int groups = (a.q_heads + U - 1) / U + 2 * ((a.kv_heads + U - 1) / U);
    const int most = kMaxThreads / L, parts = (groups + most - 1) / most;
    const int threads = ((groups + parts - 1) / parts * L + 31) / 32 * 32;
    const int resident = num_sms * std::min(32, kResident / threads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(a.rows, std::max(1, resident / parts)), parts, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<L, U, HALVES>, a);
}

template <int L>
cudaError_t launch_lanes(const RopeArgs &a, int num_sms, cudaStream_t stream, bool pdl) {
    // U = 1 for few heads in all, so that they spread over the SMs: one row of 9 heads of 128
    // 2.1 us, 2.5 with U = 4; 64 rows of 9 heads 2.7 and 3.0; 64 rows of 72, close to the
    // limit, 3.5 both; 128 rows of 72 4.3 and 3.7.
    const long long heads = static_cast<long long>(a.rows) * (a.q_heads + 2 * a.kv_heads);
    const bool halves = a.rot_dim > 0 && !a.interleaved, few = heads * L < num_sms * 512ll;
    if (halves) {
        if (few) return launch<L, 1, true>(a, num_sms, stream, pdl);
        return launch<L, 4, true>(a, num_sms, stream, pdl);
    }
    if (few) return launch<L, 1, false>(a, num_sms, stream, pdl);
    return launch<L, 4, false>(a, num_sms, stream, pdl);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs &a, int num_sms, cudaStream_t stream, bool pdl) {
    if (a.head_dim <= 64) return launch_lanes<8>(a, num_sms, stream, pdl);
    if (a.head_dim <= 128) return launch_lanes<16>(a, num_sms, stream, pdl);
    return launch_lanes<32>(a, num_sms, stream, pdl);
}

cudaError_t rope_error_word(int *value, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_rope_err, sizeof(int));
    if (e != cudaSuccess || !clear || *value == 0) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_rope_err, &zero, sizeof(int));
}

}  // namespace skinny
