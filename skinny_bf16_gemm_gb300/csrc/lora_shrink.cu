// The first half of the low-rank adapters beside a decode GEMM: t[m] = A_a x[m], a the
// adapter of row m, in FP32. The second half, scale B_a t, is in the GEMM's epilogue
// (decode_gemm.cu), which adds the K slices' sums kept here in order.
//
// Bound by HBM for many adapters (each A in use is read once), by latency for few. One CTA
// per (K slice, 16 rows of A, first row of x with the adapter): it gathers the rows of x that
// have the same adapter and multiplies 16 rows of A by up to 16 of them at a time on the
// tensor cores (mma.sync: 16 rows of A, 8 rows of x; a product of this size would not pay
// for setting up tensor memory). Rows of x that are not their adapter's first leave at once.
// The order of the K products within a 32-wide step is free, so each lane loads 16 bytes of a
// row and feeds two MMAs from them.
//
// Programmatic dependent launch: the GEMM behind this kernel may start once every CTA here
// has seen its own predecessor complete, so x is there for it, and streams its weights and
// multiplies them while this kernel runs; only its epilogue waits for the sums.
//
// Measured (in a graph, both kernels; the GEMM with its epilogue alone in brackets): 13.6 us
// (12.3) at 1 x 2048 x 7168, rank 16; 56.3 (44.9) at 16 x 18432 x 7168 with 16 adapters of rank
// 64; 61.8 (49.1) at 64 x 7168 x 18432 with 64 adapters of rank 16 (38 MB of A
// and 15 MB of B beside the 264 MB of the weight; at the copy rate these take 7.8 us).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "plan.cuh"
#include "ptx.cuh"

namespace skinny {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;     // K values of a warp's step: 16 bytes a lane
constexpr int kRankTile = 16;
constexpr int kTokens = 16;   // rows of x at a time
__device__ int g_lora_err;  // nonzero: an adapter index was out of range

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(kThreads)
    lora_shrink_kernel(const uint16_t *__restrict__ x, LoraArgs l, int M, int K, int slice) {
    __shared__ int sm_rows[kMaxM];
    __shared__ int sm_count;
    __shared__ float sm_sums[kWarps][kTokens][kRankTile];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int split = blockIdx.x, j0 = blockIdx.y * kRankTile, m = blockIdx.z;

    ptx::pdl_wait();
    ptx::pdl_launch_dependents();

    // The rows with this row's adapter; only the first of them goes on.
    if (warp == 0) {
        const int mine = __ldcg(l.adapters + m);
        const int lo = lane < M ? __ldcg(l.adapters + lane) : -1, hi = lane + 32 < M ? __ldcg(l.adapters + lane + 32) : -1;
        const bool good = mine >= 0 && mine < l.count;
        if (mine >= l.count && split == 0 && j0 == 0 && lane == 0) atomicOr(&g_lora_err, 1);
        const unsigned at_lo = __ballot_sync(0xFFFFFFFFu, lo == mine), at_hi = __ballot_sync(0xFFFFFFFFu, hi == mine);
        const bool first = (at_lo != 0 ? __ffs(at_lo) - 1 : 31 + __ffs(at_hi)) == m;
        const unsigned below = (1u << lane) - 1u;
        if (lo == mine && lane < M) sm_rows[__popc(at_lo & below)] = lane;
        if (hi == mine && lane + 32 < M) sm_rows[__popc(at_lo) + __popc(at_hi & below)] = lane + 32;
        if (lane == 0) sm_count = good && first ? __popc(at_lo) + __popc(at_hi) : 0;
    }
    __syncthreads();
    const int count = sm_count;
    if (count == 0) return;
    const int adapter = __ldcg(l.adapters + m);

    const int k_begin = split * slice, k_end = min(k_begin + slice, K);
    const int g = lane / 4, t8 = (lane & 3) * 8;
    const bool row_lo = j0 + g < l.rank, row_hi = j0 + g + 8 < l.rank;
    const uint16_t *a_lo = l.A + (static_cast<size_t>(adapter) * l.rank + j0 + (row_lo ? g : 0)) * K;
    const uint16_t *a_hi = l.A + (static_cast<size_t>(adapter) * l.rank + j0 + (row_hi ? g + 8 : 0)) * K;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // Up to 16 rows of x at a time. The steps whose loads are on their way together: 8, or 4 with
    // a second block of 8 rows.
    auto products = [&](int c0, auto second) {
        constexpr int kUnroll = second ? 4 : 8;
        const bool in0 = c0 + g < count, in1 = second && c0 + 8 + g < count;
        const uint16_t *x0 = x + static_cast<size_t>(sm_rows[in0 ? c0 + g : 0]) * K;
        const uint16_t *x1 = x + static_cast<size_t>(sm_rows[in1 ? c0 + 8 + g : 0]) * K;
        float d[2][4] = {};
        for (int k = k_begin + warp * kStep + t8; k - t8 < k_end; k += kWarps * kStep * kUnroll) {
            uint4 al[kUnroll], ah[kUnroll], b0[kUnroll], b1[second ? kUnroll : 1];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int at = k + u * kWarps * kStep;
                const bool in = at < k_end;  // K and the slices are multiples of 8
                al[u] = in && row_lo ? __ldcg(reinterpret_cast<const uint4 *>(a_lo + at)) : zero;
                ah[u] = in && row_hi ? __ldcg(reinterpret_cast<const uint4 *>(a_hi + at)) : zero;
                b0[u] = in && in0 ? __ldcg(reinterpret_cast<const uint4 *>(x0 + at)) : zero;
                if constexpr (second) b1[u] = in && in1 ? __ldcg(reinterpret_cast<const uint4 *>(x1 + at)) : zero;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                mma16816(d[0], al[u].x, ah[u].x, al[u].y, ah[u].y, b0[u].x, b0[u].y);
                mma16816(d[0], al[u].z, ah[u].z, al[u].w, ah[u].w, b0[u].z, b0[u].w);
                if constexpr (second) {
                    mma16816(d[1], al[u].x, ah[u].x, al[u].y, ah[u].y, b1[u].x, b1[u].y);
                    mma16816(d[1], al[u].z, ah[u].z, al[u].w, ah[u].w, b1[u].z, b1[u].w);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) sm_sums[warp][b * 8 + (lane & 3) * 2 + (e & 1)][g + (e >> 1) * 8] = d[b][e];
    };
    for (int c0 = 0; c0 < count; c0 += kTokens) {
        if (c0 + 8 < count)
            products(c0, std::true_type{});
        else
            products(c0, std::false_type{});
        __syncthreads();
        for (int i = tid; i < kTokens * kRankTile; i += kThreads) {
            const int token = i / kRankTile, j = i % kRankTile;
            if (c0 + token < count && j0 + j < l.rank) {
                float s = sm_sums[0][token][j];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) s += sm_sums[w][token][j];
                l.sums[(static_cast<size_t>(split) * M + sm_rows[c0 + token]) * l.rank + j0 + j] = s;
            }
        }
        __syncthreads();
    }
}

}  // namespace

// K slices of a call: of 256 values, or more where that would be more than 32 of them, than about
// eight CTAs an SM if every row had an adapter of its own, or than the scratch has room for (of fewer
// where K is no multiple: K = 264 two of 136 and 128).
int lora_splits(int M, int K, int rank, int num_sms) {
    const int tiles = (rank + kRankTile - 1) / kRankTile;
    int s = (K + 255) / 256;
    const int most = 8 * num_sms / (M * tiles), room = kLoraScratchFloats / (M * rank);
    s = s < 32 ? s : 32;
    s = s < most ? s : most;
    s = s < room ? s : room;
    return s > 1 ? s : 1;
}

cudaError_t launch_lora_shrink(const void *x, const LoraArgs &l, int M, int K, int num_sms, cudaStream_t stream,
                               bool pdl) {
    // Slices of whole steps of 8 values; the last ones may be empty.
    const int slice = ((K + l.splits - 1) / l.splits + 7) / 8 * 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.splits, (l.rank + kRankTile - 1) / kRankTile, M);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // Many CTAs that wait for the kernel before take its place: 64 x 7168 x 18432 with 64 adapters
    // of rank 16 67 us, 61 without; few ones are ready sooner (1 x 2048 x 7168 12.4 us, 13.6).
    const long long ctas = static_cast<long long>(cfg.gridDim.x) * cfg.gridDim.y * cfg.gridDim.z;
    cfg.numAttrs = pdl && ctas <= 2 * num_sms ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, lora_shrink_kernel, static_cast<const uint16_t *>(x), l, M, K, slice);
}

cudaError_t lora_error_word(int **word) { return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_lora_err); }

}  // namespace skinny
