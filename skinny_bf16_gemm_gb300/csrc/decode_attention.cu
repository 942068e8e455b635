// Attention of one new token per row over a paged key-value cache on GB300 (sm_103a).
//
//   s_j = scale q.k_j,  m = max s_j,  l = sum exp(s_j - m),  o = sum exp(s_j - m) v_j / l
// over the tokens j the row sees: all before its length, or with a sliding window
// the last `window` of them and the first `sinks`. One pass over the cache with the
// running maximum and sum; the query heads that share a key head are done together,
// so every key and value is read once. Bound by HBM: 4 D bytes a token and key head
// against 4 G D flops (G heads sharing) -- 8 flops a byte for G = 8.
//
// CTAs of 4 warps, two to an SM (one for heads over 128), take equal ranges of
// 64-token tiles (attention_plan.cuh). A warp streams its own 16 tokens of every
// tile through a private ring of cp.async stages and keeps its own maximum, sum and
// accumulator, so nothing in the main loop waits for another warp; the four are
// joined when the piece of an item ends. The ring is filled by 16-byte copies with
// each token's address from the block table, so pages of any size, tokens at any
// 16-byte-aligned strides and ranges that end inside a page are all the same to it;
// rows are padded by 16 bytes, which spreads ldmatrix over the banks.
// The products run on the tensor cores with tokens (scores) and head dimension
// (output) as the MMA's 16 rows and the query heads as its 8 columns: HBM feeds an
// SM about 23 bytes a clock, a fraction of what these small MMAs need to be fast.
// Weights p are split into two BF16 terms (p truncated, and the rest rounded: within
// 2^-15 of p), so the product with V loses nothing that the BF16 output shows; maxima
// and sums are FP32.
//
// An item whose tiles span several CTAs is joined by whichever of them is last to
// publish its partial (a counter in the workspace): it adds the partials in range
// order, so the bits do not depend on who was last. More than 16 partials are joined
// in two such levels, 16 at a time, to keep the last reader's share short. No CTA
// waits for another.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "attention_plan.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace skinny {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 16;  // tokens of a warp's stage
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kAttnMaxJoin = 24;  // partials of one join: kAttnGroup, or the groups of the largest grid
__device__ int g_attn_err;  // nonzero: a length or page index was out of range

template <int D, int NB>
struct Shape {
    static constexpr int kCtasPerSm = D <= 128 ? 2 : 1;
    static constexpr int kRowBytes = D * 2 + 16;
    static constexpr int kStageBytes = 2 * kSub * kRowBytes;  // keys, then values
    static constexpr int kStages = D <= 64 ? 5 : D <= 96 ? 4 : D <= 128 ? 3 : D <= 192 ? 4 : 3;
    static constexpr int kHeads = 8 * NB;
    static constexpr int kMergeStride = D + 4;  // floats: spreads the fragment stores over the banks
    static constexpr int kRingBytes = kStages * kStageBytes;
    static constexpr int kMlOffset = kWarps * kRingBytes;           // [kWarps][kHeads] m, then l
    static constexpr int kScaleOffset = kMlOffset + 2 * kWarps * kHeads * 4;  // [kAttnMaxJoin][kHeads]
    static constexpr int kPrefixOffset = kScaleOffset + kAttnMaxJoin * kHeads * 4;
    static_assert(kHeads * kMergeStride * 4 <= kRingBytes, "a warp's accumulator reuses its ring");
    static int bytes(int rows) { return kPrefixOffset + (rows + 1 + 8) * 4; }
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool full) {
    const int bytes = full ? 16 : 0;  // 0: the 16 bytes are zero-filled, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// d (16 x 8) += a (16 x 16) b (16 x 8), BF16 products, FP32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return static_cast<uint32_t>(__bfloat16_as_ushort(b.x)) |
           (static_cast<uint32_t>(__bfloat16_as_ushort(b.y)) << 16);
}

// What truncating a weight p >= 0 to BF16 leaves. Never zero: both terms of a weight
// stay positive, so that an infinite value comes out infinite and not 0 * inf or
// inf - inf. 2^-126 is below half a step of any p above 2^-118.
__device__ __forceinline__ float rest_of(float p) {
    return fmaxf(p - __uint_as_float(__float_as_uint(p) & 0xFFFF0000u), 1.17549435e-38f);
}

// Tokens a row of length n sees, and what lies between its sinks and its window.
struct Seen {
    int count;  // tokens seen
    int sinks;  // those before the gap
    int gap;    // tokens skipped after them
};
__device__ __forceinline__ Seen seen_of(int n, int window, int sinks) {
    Seen s = {n, n, 0};
    if (window > 0 && n > window) {
        s.sinks = min(sinks, n - window);
        s.gap = n - window - s.sinks;
        s.count = n - s.gap;
    }
    return s;
}

// Ranges of the tile sequence: the first `extra` of `ctas` CTAs take base + 1 tiles.
struct Ranges {
    int ctas, base, extra;
    __device__ int begin(int c) const { return c * base + min(c, extra); }
    __device__ int owner(int x) const {
        const int cut = extra * (base + 1);
        return x < cut ? x / (base + 1) : extra + (x - cut) / base;
    }
};

template <int D, int NB>
__global__ void __launch_bounds__(kThreads, Shape<D, NB>::kCtasPerSm)
    decode_attention_kernel(const AttentionArgs a) {
    using S = Shape<D, NB>;
    constexpr int kChunks = D / 8;            // 16-byte chunks of a token's row
    constexpr int kCopies = kSub * kChunks / 32;
    constexpr int kSteps = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    float *sm_m = reinterpret_cast<float *>(smem + S::kMlOffset);
    float *sm_l = sm_m + kWarps * S::kHeads;
    float *sm_scale = reinterpret_cast<float *>(smem + S::kScaleOffset);
    int *prefix = reinterpret_cast<int *>(smem + S::kPrefixOffset);
    int *sm_tmp = prefix + a.rows + 1;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

    ptx::pdl_launch_dependents();
    ptx::pdl_wait();

    // Prefix sums of the rows' tiles. A length is taken within [0, capacity].
    const int per = (a.rows + kThreads - 1) / kThreads;
    const int r_lo = min(tid * per, a.rows), r_hi = min(r_lo + per, a.rows);
    auto row_length = [&](int r) {
        int n = __ldcg(a.lengths + r);
        if (n < 0 || n > a.capacity) {
            if (blockIdx.x == 0) atomicOr(&g_attn_err, 1);
            n = n < 0 ? 0 : a.capacity;
        }
        return n;
    };
    int mine = 0;
    for (int r = r_lo; r < r_hi; ++r) {
        const int n = seen_of(row_length(r), a.window, a.sinks).count;
        mine += (n + kAttnTile - 1) / kAttnTile;
        prefix[r + 1] = mine;
    }
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) sm_tmp[warp] = scan;
    __syncthreads();
    int before = scan - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) before += sm_tmp[w];
    for (int r = r_lo; r < r_hi; ++r) prefix[r + 1] += before;
    if (tid == 0) prefix[0] = 0;
    __syncthreads();

    // Rows that see nothing: zeros, and a log-sum of -inf.
    for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
        if (prefix[r + 1] != prefix[r]) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + static_cast<size_t>(r) * a.q_heads * D);
        for (int i = tid; i < a.q_heads * kChunks; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr)
            for (int h = tid; h < a.q_heads; h += kThreads)
                a.lse[static_cast<size_t>(r) * a.q_heads + h] = -INFINITY;
    }

    const int items_per_row = a.kv_heads * a.head_blocks;
    const int total = prefix[a.rows] * items_per_row;  // below 2^31 (host check)
    if (total == 0) return;
    Ranges rg;
    rg.ctas = min(static_cast<int>(gridDim.x), total);
    if (static_cast<int>(blockIdx.x) >= rg.ctas) return;
    rg.base = total / rg.ctas;
    rg.extra = total - rg.base * rg.ctas;
    const int cta = blockIdx.x;
    int x = rg.begin(cta);
    const int x_end = rg.begin(cta + 1);

    int row = 0;  // the row of tile x: the last one whose first tile is at or before it
    for (int lo = 0, hi = a.rows; lo < hi;) {
        const int mid = (lo + hi) / 2;
        if (prefix[mid + 1] * items_per_row <= x) lo = mid + 1; else hi = mid;
        row = lo;
    }

    const uint32_t ring = sbase + warp * S::kRingBytes;
    float *merge = reinterpret_cast<float *>(smem + warp * S::kRingBytes);
    __shared__ uint32_t sm_valid[kWarps][S::kStages];
    __shared__ int sm_last;

    while (x < x_end) {
        while (prefix[row + 1] * items_per_row <= x) ++row;
        const int row_tiles = prefix[row + 1] - prefix[row];
        const int in_row = x - prefix[row] * items_per_row;
        const int item = in_row / row_tiles;
        const int tile0 = in_row - item * row_tiles;
        const int tile1 = min(row_tiles, tile0 + x_end - x);
        const int kv_head = item / a.head_blocks;
        const int g0 = (item - kv_head * a.head_blocks) * a.block_heads;  // first head of the group
        const int n_heads = min(a.block_heads, a.group - g0);
        const int head0 = kv_head * a.group + g0;
        const int length = min(max(__ldcg(a.lengths + row), 0), a.capacity);
        const Seen seen = seen_of(length, a.window, a.sinks);
        const int *table = a.block_table + static_cast<size_t>(row) * a.table_stride;
        const uint16_t *kbase = a.k + kv_head * a.head_stride;
        const uint16_t *vbase = a.v + kv_head * a.head_stride;

        // This warp's stages: tokens [t0, t0 + 16) of every tile of the piece.
        const int n_stages = tile1 - tile0;
        auto issue = [&](int i) {  // stage i of the piece into the ring
            if (i < n_stages) {
                const int t = (tile0 + i) * kAttnTile + warp * kSub + (lane & 15);
                long long off = -1;
                if (t < seen.count) {
                    const int j = t < seen.sinks ? t : t + seen.gap;
                    const int entry = j / a.page_size;
                    const int page = __ldcg(table + entry);
                    if (page >= 0 && page < a.num_pages)
                        off = page * a.page_stride + static_cast<long long>(j - entry * a.page_size) * a.token_stride;
                    else
                        atomicOr(&g_attn_err, 1);
                }
                const uint32_t valid = __ballot_sync(0xFFFFFFFFu, off >= 0);
                if (lane == 0) sm_valid[warp][i % S::kStages] = valid;
                const uint32_t st = ring + (i % S::kStages) * S::kStageBytes;
#pragma unroll
                for (int it = 0; it < kCopies; ++it) {
                    const int id = it * 32 + lane, tok = id / kChunks, ch = id % kChunks;
                    const long long o = __shfl_sync(0xFFFFFFFFu, off, tok);
                    const uint32_t dst = st + tok * S::kRowBytes + ch * 16;
                    const long long e = (o < 0 ? 0 : o) + ch * 8;
                    cp_async16(dst, kbase + e, o >= 0);
                    cp_async16(dst + kSub * S::kRowBytes, vbase + e, o >= 0);
                }
            }
            cp_async_commit();  // an empty group past the end keeps the count
        };
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) issue(i);

        // Queries as the MMA's B: head lane / 4 of each block of 8, values 2 (lane % 4) on.
        uint32_t qf[kSteps][NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int h = b * 8 + lane / 4;
            const uint16_t *q = a.q + row * a.q_stride + static_cast<long long>(head0 + h) * D + (lane & 3) * 2;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                qf[ks][b][0] = h < n_heads ? __ldcg(reinterpret_cast<const unsigned *>(q + ks * 16)) : 0u;
                qf[ks][b][1] = h < n_heads ? __ldcg(reinterpret_cast<const unsigned *>(q + ks * 16 + 8)) : 0u;
            }
        }

        float o[kSteps][NB][4];
        float m[NB][2], l[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            m[b][0] = m[b][1] = -INFINITY;
            l[b][0] = l[b][1] = 0.0f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[s][b][i] = 0.0f;
        }

        for (int i = 0; i < n_stages; ++i) {
            cp_async_wait<S::kStages - 2>();
            __syncwarp();
            issue(i + S::kStages - 1);  // into the stage read last time round
            const uint32_t st = ring + (i % S::kStages) * S::kStageBytes;
            const uint32_t valid = sm_valid[warp][i % S::kStages];

            // Scores: rows = tokens lane / 4 and + 8, columns = heads 2 (lane % 4) and + 1.
            float c[NB][4] = {};
            {
                const uint32_t at = st + ((lane & 7) + ((lane >> 3) & 1) * 8) * S::kRowBytes + (lane >> 4) * 16;
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) {
                    uint32_t kf[4];
                    ldmatrix4(kf, at + ks * 32);
#pragma unroll
                    for (int b = 0; b < NB; ++b) mma16816(c[b], kf, qf[ks][b][0], qf[ks][b][1]);
                }
            }
            const bool v0 = (valid >> (lane / 4)) & 1, v1 = (valid >> (lane / 4 + 8)) & 1;
            float top[NB][2];
            bool grew = false;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    c[b][e] = v0 ? c[b][e] * a.scale_log2 : -INFINITY;
                    c[b][e + 2] = v1 ? c[b][e + 2] * a.scale_log2 : -INFINITY;
                    float t = fmaxf(c[b][e], c[b][e + 2]);
                    t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
                    top[b][e] = fmaxf(t, m[b][e]);
                    grew |= top[b][e] > m[b][e];
                }
            }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // A maximum that is still -inf leaves zeros: any factor will do.
                        const float f = m[b][e] == -INFINITY ? 0.0f : exp2_approx(m[b][e] - top[b][e]);
                        m[b][e] = top[b][e];
                        l[b][e] *= f;
#pragma unroll
                        for (int s = 0; s < kSteps; ++s) {
                            o[s][b][e] *= f;
                            o[s][b][e + 2] *= f;
                        }
                    }
            }
            uint32_t hi[NB][2], lo[NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float ref = m[b][e & 1] == -INFINITY ? 0.0f : m[b][e & 1];
                    p[e] = exp2_approx(c[b][e] - ref);
                    l[b][e & 1] += p[e];
                }
                // Tokens by heads -> heads by tokens, the B operand of the product with V.
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t h = __byte_perm(__float_as_uint(p[2 * e]), __float_as_uint(p[2 * e + 1]), 0x7632);
                    const uint32_t r = pack_bf16(rest_of(p[2 * e]), rest_of(p[2 * e + 1]));
                    hi[b][e] = movmatrix_trans(h);
                    lo[b][e] = movmatrix_trans(r);
                }
            }
            {
                const uint32_t at = st + kSub * S::kRowBytes +
                                    ((lane & 7) + ((lane >> 4) & 1) * 8) * S::kRowBytes + ((lane >> 3) & 1) * 16;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    uint32_t vf[4];
                    ldmatrix4_trans(vf, at + s * 32);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        mma16816(o[s][b], vf, hi[b][0], hi[b][1]);
                        mma16816(o[s][b], vf, lo[b][0], lo[b][1]);
                    }
                }
            }
            __syncwarp();  // every lane is done with the stage before it is refilled
        }
        cp_async_wait<0>();
        __syncwarp();

        // ---- join the four warps ----
        // Sums over the lanes that share a column; the maxima are equal there already.
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[b][e] += __shfl_xor_sync(0xFFFFFFFFu, l[b][e], 4);
                l[b][e] += __shfl_xor_sync(0xFFFFFFFFu, l[b][e], 8);
                l[b][e] += __shfl_xor_sync(0xFFFFFFFFu, l[b][e], 16);
                if (lane < 4) {
                    sm_m[warp * S::kHeads + b * 8 + lane * 2 + e] = m[b][e];
                    sm_l[warp * S::kHeads + b * 8 + lane * 2 + e] = l[b][e];
                }
            }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    merge[(b * 8 + (lane & 3) * 2 + (i & 1)) * S::kMergeStride + s * 16 + lane / 4 + (i >> 1) * 8] =
                        o[s][b][i];
        __syncthreads();

        // Piece q of n of this item: CTAs first .. first + n - 1 hold one each.
        const int item_x0 = prefix[row] * items_per_row + item * row_tiles;
        const int first = rg.owner(item_x0);
        const int pieces = rg.owner(item_x0 + row_tiles - 1) - first + 1;
        const int slot = 2 * cta + (tile0 > 0 ? 0 : 1);

        // Head h's values over n sources: combined maximum and sum, and each source's
        // factor in sm_scale.
        auto store_out = [&](int h, int d4, float4 v, float inv) {
            const uint2 w = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
            *reinterpret_cast<uint2 *>(a.out + (static_cast<size_t>(row) * a.q_heads + head0 + h) * D + d4 * 4) = w;
        };
        auto store_lse = [&](int h, float mm, float ll) {
            if (a.lse != nullptr)
                a.lse[static_cast<size_t>(row) * a.q_heads + head0 + h] =
                    ll > 0.0f || ll != ll ? (mm + log2f(ll)) * kLn2 : -INFINITY;
        };

        constexpr int kQuads = D / 4;
        float *ws_slot = a.partials + static_cast<size_t>(slot) * kAttnSlotFloats;
        for (int i = tid; i < n_heads * kQuads; i += kThreads) {
            const int h = i / kQuads, d4 = i % kQuads;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w * S::kHeads + h]);
            const float ref = mm == -INFINITY ? 0.0f : mm;
            float ll = 0.0f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2_approx(sm_m[w * S::kHeads + h] - ref);
                const float4 u = *reinterpret_cast<const float4 *>(
                    reinterpret_cast<const float *>(smem + w * S::kRingBytes) + h * S::kMergeStride + d4 * 4);
                ll += f * sm_l[w * S::kHeads + h];
                v.x += f * u.x; v.y += f * u.y; v.z += f * u.z; v.w += f * u.w;
            }
            if (pieces == 1) {
                store_out(h, d4, v, ll == 0.0f ? 0.0f : __fdiv_rn(1.0f, ll));
                if (d4 == 0) store_lse(h, mm, ll);
            } else {
                __stcg(reinterpret_cast<float4 *>(ws_slot + h * D + d4 * 4), v);
                if (d4 == 0) {
                    __stcg(ws_slot + 4096 + h, mm);
                    __stcg(ws_slot + 4096 + kAttnMaxHeads + h, ll);
                }
            }
        }

        if (pieces > 1) {
            // Arrive; the last of the group joins it, and the last group's joiner the
            // groups. Counters go back to zero for the next call.
            const int me = cta - first;
            const int group = me / kAttnGroup;
            const int groups = (pieces + kAttnGroup - 1) / kAttnGroup;
            auto slot_of = [&](int q) { return 2 * (first + q) + (q == 0 ? 1 : 0); };
            auto arrive = [&](unsigned *counter, int expected) -> bool {
                __syncthreads();  // every thread's partial is stored
                if (tid == 0) {
                    __threadfence();
                    const unsigned old = atomicAdd(counter, 1u);
                    sm_last = old + 1 == static_cast<unsigned>(expected);
                    if (sm_last) *counter = 0u;
                    __threadfence();
                }
                __syncthreads();
                return sm_last != 0;
            };
            // Join sources q0, q0 + step, .. (n of them) into `dst` slot, or the output.
            auto join = [&](int q0, int step, int n, int dst) {
                float mm = -INFINITY, ll = 0.0f;
                if (tid < n_heads) {
                    for (int k = 0; k < n; ++k)
                        mm = fmaxf(mm, __ldcg(a.partials + static_cast<size_t>(slot_of(q0 + k * step)) * kAttnSlotFloats +
                                              4096 + tid));
                    const float ref = mm == -INFINITY ? 0.0f : mm;
                    for (int k = 0; k < n; ++k) {
                        const float *src = a.partials + static_cast<size_t>(slot_of(q0 + k * step)) * kAttnSlotFloats + 4096;
                        const float f = exp2_approx(__ldcg(src + tid) - ref);
                        ll += f * __ldcg(src + kAttnMaxHeads + tid);
                        sm_scale[k * S::kHeads + tid] = f;
                    }
                    sm_m[tid] = mm;
                    sm_l[tid] = ll;
                }
                __syncthreads();
                float *to = a.partials + static_cast<size_t>(dst < 0 ? 0 : dst) * kAttnSlotFloats;
                for (int i = tid; i < n_heads * kQuads; i += kThreads) {
                    const int h = i / kQuads, d4 = i % kQuads;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k = 0; k < n; ++k) {
                        const float f = sm_scale[k * S::kHeads + h];
                        const float4 u = __ldcg(reinterpret_cast<const float4 *>(
                            a.partials + static_cast<size_t>(slot_of(q0 + k * step)) * kAttnSlotFloats + h * D + d4 * 4));
                        v.x += f * u.x; v.y += f * u.y; v.z += f * u.z; v.w += f * u.w;
                    }
                    if (dst < 0) {
                        const float sum = sm_l[h];
                        store_out(h, d4, v, sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum));
                        if (d4 == 0) store_lse(h, sm_m[h], sum);
                    } else {
                        __stcg(reinterpret_cast<float4 *>(to + h * D + d4 * 4), v);
                        if (d4 == 0) {
                            __stcg(to + 4096 + h, sm_m[h]);
                            __stcg(to + 4096 + kAttnMaxHeads + h, sm_l[h]);
                        }
                    }
                }
            };
            const int q0 = group * kAttnGroup;
            const int in_group = min(kAttnGroup, pieces - q0);
            const bool one_level = groups == 1;
            if (arrive(a.counters + 2 * slot_of(q0), in_group)) {
                join(q0, 1, in_group, one_level ? -1 : slot_of(q0));
                if (!one_level && arrive(a.counters + 2 * slot_of(0) + 1, groups)) join(0, kAttnGroup, groups, -1);
            }
        }
        __syncthreads();  // the ring and the joins' arrays are reused
        x += tile1 - tile0;
    }
}

template <int D, int NB>
cudaError_t launch(const AttentionArgs &a, int num_sms, int device, cudaStream_t stream, bool pdl) {
    using S = Shape<D, NB>;
    static int configured[64] = {};
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    const int most = S::bytes(kAttnMaxRows);
    if (!configured[device]) {
        cudaError_t e = cudaFuncSetAttribute(decode_attention_kernel<D, NB>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        configured[device] = 1;
    }
    // No more CTAs than the tables could ever hold tiles.
    const long long tiles = static_cast<long long>(a.rows) * a.kv_heads * a.head_blocks *
                            ((a.capacity + kAttnTile - 1ll) / kAttnTile);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::max(1ll, std::min<long long>(num_sms * S::kCtasPerSm, tiles))), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = S::bytes(a.rows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, decode_attention_kernel<D, NB>, a);
}

template <int D>
cudaError_t launch_dim(const AttentionArgs &a, int num_sms, int device, cudaStream_t stream, bool pdl) {
    if (a.block_heads <= 8) return launch<D, 1>(a, num_sms, device, stream, pdl);
    if (a.block_heads <= 16) return launch<D, 2>(a, num_sms, device, stream, pdl);
    if constexpr (D <= 128) return launch<D, 4>(a, num_sms, device, stream, pdl);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decode_attention(const AttentionArgs &a, int head_dim, int num_sms, int device,
                                    cudaStream_t stream, bool pdl) {
    switch (head_dim) {
        case 64: return launch_dim<64>(a, num_sms, device, stream, pdl);
        case 96: return launch_dim<96>(a, num_sms, device, stream, pdl);
        case 128: return launch_dim<128>(a, num_sms, device, stream, pdl);
        case 192: return launch_dim<192>(a, num_sms, device, stream, pdl);
        case 256: return launch_dim<256>(a, num_sms, device, stream, pdl);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t attention_error_word(int *value, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_attn_err, sizeof(int));
    if (e != cudaSuccess || !clear || *value == 0) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_attn_err, &zero, sizeof(int));
}

}  // namespace skinny
