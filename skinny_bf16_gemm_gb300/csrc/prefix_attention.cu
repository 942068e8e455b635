// Attention of all rows of a decode batch over a prefix that they share, on GB300 (sm_103a):
// the part of decode_attention_shared_prefix_bf16 that is computed once for all, and the
// join with the rows' own tokens.
//
//   s_ij = scale q_i.k_j,  m_i = max_j s_ij,  l_i = sum_j exp(s_ij - m_i),
//   o_i = sum_j exp(s_ij - m_i) v_j      over the prefix's tokens j
// for the query rows i of a key head: every row's heads that share it (prefix_plan.cuh). All of
// them go through the prefix at the same time, so that it is read once; from some 300 query
// rows on the tensor cores are the bound, below it HBM.
//
// A CTA has one or two tiles of 128 query rows in shared memory and a ring of tiles of the
// prefix's keys and values, in turn. Roles:
//   warps 0-3 (4-7)   softmax of the first (second) tile: thread = query row = TMEM lane;
//   4 loader warps    the ring, in the 128-byte swizzle that the MMA's descriptors name: by TMA
//                     boxes of as many tokens as pages and tiles both are multiples of, or,
//                     for pages of no multiple of 8 and for a tile that the prefix ends in
//                     (what is behind its end must come out as zeros), by 16-byte cp.async
//                     with each token's address. Two for the keys, two for the values: a
//                     thread takes some 200 clocks to issue a box, of whatever size, and the
//                     threads of a warp take turns;
//   2 MMA warps a tile  the scores, S = Q K^T, from shared memory (both K-major) into tensor
//                     memory; and O += P V, P in tensor memory and V as it lies, MN-major.
// Scores, weights and output have places of their own in tensor memory: a softmax thread takes
// its row of scores into registers and sets their place free, so that the next step's are
// computed while it works, and the two tiles' softmaxes and products fill each other's gaps.
// The maximum is kept until a score is 2^8 past it; only then O is rescaled, by the softmax
// threads, in tensor memory. P is rounded to BF16 (to nearest: within 2^-8 of each weight):
// the roundings of different tokens are independent, so they average out in o as the weights
// do, and add at most as much as the output's own rounding. A second BF16 term, as
// decode_attention_bf16 has where the products are free, would cost half the tensor time
// again with two tiles, and lengthen the softmax and the products, which take turns, with one.
// Maxima, sums and o are FP32.
//
// Measured (in a graph, with the own tokens and the join): 151 us for 64 rows x 56 heads over 8
// behind 65521 tokens with 1000 of their own each, of 62 us that the products take at the peak
// rate (decode_attention_bf16 over joined tables: 2107 us); this kernel alone is 104 us, some 2100
// clocks a step of 80 tokens of which the tensor cores are busy for 1280. Their operands are the
// closer bound: 144 KB read from shared memory and 40 KB of new tiles written a step are 1440
// clocks at 128 bytes each, the queries the larger part (64 KB), which tensor memory has no room
// for. It is not the softmax: two threads a row, half the scores each, took 10 us more, and
// 3-4 % less with one tile of query rows. 22.5 us for 64 rows x 7 heads behind 16001
// tokens with 1000 of their own, side by side (prefix_plan.cuh prefix_ctas).
//
// Every wait is bounded; one that runs out is recorded, the CTA waits for its own copies and
// MMAs, frees its tensor memory and ends.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "prefix_plan.cuh"
#include "ptx.cuh"

namespace skinny {
namespace {

constexpr float kNoMaximum = -3.402823466e+38f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr uint64_t kDrainLimitNs = 200000000ull;   // 0.2 s for work already issued
constexpr int kErrWait = 1, kErrRange = 2, kErrLeft = 4;
// kErrWait: a wait ran out; kErrRange: a length or page out of range; kErrLeft: a CTA that gave up
// ended before its own copies and products were seen to be complete
__device__ int g_prefix_err;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp_async16_or_zeros(uint32_t dst, const void *src, bool full) {
    const int bytes = full ? 16 : 0;  // 0: the 16 bytes are zero-filled, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
// Two FP32 operations an instruction.
__device__ __forceinline__ void fma2(float &x, float &y, float c, float d) {
    asm("{\n\t.reg .b64 a, b, e;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 e, {%3, %3};\n\t"
        "fma.rn.f32x2 a, a, b, e;\n\tmov.b64 {%0, %1}, a;\n\t}" : "+f"(x), "+f"(y) : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float &x, float &y, float c, float d) {
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}" : "+f"(x), "+f"(y) : "f"(c), "f"(d));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

constexpr int kMaskRing = 16;  // tiles whose masks are kept: more than the loader is ahead

template <int D, int NT>
struct Shape {
    static constexpr int kTokens = prefix_tokens(D, NT);
    static constexpr int kChunks = (D + 63) / 64;               // 128-byte chunks of a row
    static constexpr int kUnitBytes = kChunks * kTokens * 128;  // a tile's keys, or values
    static constexpr bool kMerged = prefix_merged(D);
    static constexpr int kGroupBytes = kMerged ? kChunks * 1024 : 1024;          // from 8 tokens to the next
    static constexpr int kChunkBytes = kMerged ? 1024 : kTokens * 128;           // from chunk to chunk
    static constexpr int kQChunkBytes = kPrefixRows * 128;
    static constexpr int kQBytes = kChunks * kQChunkBytes;      // one tile of queries
    static constexpr int kMiscBytes = 768;
    static constexpr int kStages = std::min(8, (232448 - 1024 - kMiscBytes - NT * kQBytes) / kUnitBytes);
    using Ring = PrefixRing<kStages>;
    // cp.async: a warp's units (of its kind) whose copies are on their way; fewer than its kind's
    // stages, so that the one that is waited for is not among them.
    static constexpr int kLag = std::max(1, kStages / 4);
    static_assert(kLag < Ring::kValues, "no unit waits for one behind it");
    static_assert(kStages >= 4, "a key and a value tile in use while others are on their way");
    static constexpr int kRingOffset = NT * kQBytes;
    static constexpr int kMaskWords = (kTokens + 31) / 32;
    static constexpr int kMaskOffset = kRingOffset + kStages * kUnitBytes;  // [kMaskRing][kMaskWords]
    static constexpr int kBarOffset = kMaskOffset + kMaskRing * kMaskWords * 4;
    static constexpr int kBars = 2 * kStages + 2 * 5 + 1;
    static constexpr int kTailOffset = kBarOffset + kBars * 8;  // tensor memory base, abort flag, units begun
    static constexpr int kBytes = kTailOffset + 24;
    static constexpr int kDynamicBytes = kBytes + 1024;  // slack to align the base to 1024
    static_assert(kDynamicBytes <= 232448, "shared memory of a CTA");
    static constexpr int kLoaders = 2;  // warps for the keys, and for the values
    static constexpr int kLoaderWarp = NT * 4, kScoresWarp = kLoaderWarp + 2 * kLoaders, kValuesWarp = kScoresWarp + NT;
    static constexpr int kThreads = (NT * 4 + 8) * 32;  // groups of four warps, the last not full
    // Registers a thread: a row of scores is kept in them. The groups of four warps have 128 each
    // (one tile: 168) at the launch; the softmax takes what the others give.
    static constexpr int kLaunchRegisters = NT == 2 ? 128 : 168, kGroups = NT + 2;
    static constexpr int kSoftmaxRegisters = NT == 2 ? 176 : 216, kOtherRegisters = NT == 2 ? 80 : 144;
    static_assert(NT * kSoftmaxRegisters + 2 * kOtherRegisters <= kGroups * kLaunchRegisters, "registers of the block");
    // Tensor memory: scores, weights and output of each tile.
    static constexpr int kPCol = NT * kTokens, kOCol = kPCol + NT * (kTokens / 2);
    static constexpr int kTmemCols = kOCol + NT * D <= 256 ? 256 : 512;
    static_assert(kOCol + NT * D <= 512, "tensor memory");
};

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1)
    prefix_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                            const PrefixArgs a) {
    using S = Shape<D, NT>;
    using Ring = typename S::Ring;
    constexpr int kTokens = S::kTokens, kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = ptx::smem_addr(smem);
    const uint32_t bar_full = sbase + S::kBarOffset;     // + 8 stage
    const uint32_t bar_empty = bar_full + 8 * kStages;   // + 8 stage
    const uint32_t bar_q = bar_empty + 8 * kStages;      // + 8 tile: the queries are there
    const uint32_t bar_s = bar_q + 16;                   // + 8 tile: a step's scores are there
    const uint32_t bar_free = bar_s + 16;                // + 8 tile: they are read
    const uint32_t bar_p = bar_free + 16;                // + 8 tile: its weights are there
    const uint32_t bar_pv = bar_p + 16;                  // + 8 tile: O has its product
    const uint32_t bar_drain = bar_pv + 16;
    volatile uint32_t *tail = reinterpret_cast<volatile uint32_t *>(smem + S::kTailOffset);
    volatile uint32_t *abort_flag = tail + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, S::kLoaders);
            ptx::mbar_init(bar_empty + 8 * s, NT);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar_q + 8 * i, 4);  // warps
            ptx::mbar_init(bar_s + 8 * i, 2);  // the products, and the issuer (the mask is there)
            ptx::mbar_init(bar_free + 8 * i, 4);
            ptx::mbar_init(bar_p + 8 * i, 4);
            ptx::mbar_init(bar_pv + 8 * i, 1);
        }
        ptx::mbar_init(bar_drain, 2 * NT);
        *abort_flag = 0u;
        ptx::fence_barrier_init();
    }
    if (warp == S::kLoaderWarp && lane == 0 && a.box_rows > 0) {
        ptx::prefetch_tensormap(&k_map);
        ptx::prefetch_tensormap(&v_map);
    }
    if (warp == S::kScoresWarp) {
        ptx::tmem_alloc(sbase + S::kTailOffset, S::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = tail[0];

    // The kernels behind this one may start once what is before it is complete: the rows' own
    // tokens do not wait for the prefix.
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();

    int length = __ldcg(a.length);
    if (length < 0 || length > a.capacity) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_prefix_err, kErrRange);
        length = length < 0 ? 0 : a.capacity;
    }
    const int steps = (length + kTokens - 1) / kTokens;  // of a key head
    const int total = steps * a.kv_heads;                // below 2^31 (host check)
    const PrefixCut cut(total, a.ranges);
    // This CTA's range of tiles, and the blocks that it goes through it for: lane, lane + lanes, ..
    const int range = blockIdx.x / a.lanes, lane_block = blockIdx.x - range * a.lanes;
    const int x_begin = range < cut.ranges ? cut.begin(range) : 0;
    const int x_end = range < cut.ranges ? cut.begin(range + 1) : 0;
    const int query_rows = a.rows * a.group;

    // Wait for the phase of a barrier with this parity; false: aborted.
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = ptx::global_timer_ns();
        for (uint32_t spin = 1;; ++spin) {
            if (ptx::mbar_try_wait(bar, parity)) return true;
            if ((spin & 15u) == 0) {
                if (*abort_flag) return false;
                if (ptx::global_timer_ns() - t0 > a.wait_limit_ns) {
                    atomicOr(&g_prefix_err, kErrWait);
                    *abort_flag = 1u;
                    return false;
                }
            }
        }
    };
    // One arrival for a warp, behind all its lanes.
    auto warp_arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar);
    };
    auto warp_wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
    // The token of a tile and its page: its element offset within the keys, or -1.
    auto place = [&](int head, int token) -> long long {
        if (token >= length) return -1;
        const int e = a.page_shift >= 0 ? token >> a.page_shift : token / a.page_size;
        const int page = __ldcg(a.table + e);
        if (page < 0 || page >= a.num_pages) return -1;
        return page * a.page_stride + (token - e * a.page_size) * a.token_stride + head * a.head_stride;
    };
    // The mask words of a tile whose tokens are all there.
    auto whole_mask = [](int i) { return kTokens - i * 32 >= 32 ? 0xFFFFFFFFu : (1u << (kTokens - i * 32) % 32) - 1u; };
    // The part of this CTA's range in one key head, for one block; in the order of blocks, then
    // key heads.
    struct Segment {
        int block, head, q0, tiles, t, n;  // first query row, tiles of query rows, first tile, steps
    };
    auto segment = [&](int block, int x) {
        Segment s;
        s.block = block;
        s.head = x / steps;
        s.q0 = block * NT * kPrefixRows;
        s.tiles = NT == 2 && query_rows - s.q0 > kPrefixRows ? 2 : 1;
        s.t = x - s.head * steps;
        s.n = min(steps - s.t, x_end - x);
        return s;
    };
    // All segments in turn: f(segment) until it is false.
    auto segments = [&](auto &&f) {
        for (int block = lane_block; block < a.blocks; block += a.lanes)
            for (int x = x_begin; x < x_end;) {
                const Segment s = segment(block, x);
                if (!f(s)) return;
                x += s.n;
            }
    };
    if (warp < S::kLoaderWarp) {
        // ---------------- softmax: thread = query row ----------------
        ptx::take_registers<S::kSoftmaxRegisters>();
        const int tile = warp / 4;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16);
        const uint32_t s_addr = lanes + tile * kTokens, p_addr = lanes + S::kPCol + tile * (kTokens / 2);
        const uint32_t o_addr = lanes + S::kOCol + tile * D;
        const float c = fabsf(a.scale_log2);
        const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;  // of the queries' signs
        const uint32_t *masks = reinterpret_cast<const uint32_t *>(smem + S::kMaskOffset);
        uint32_t count = 0;       // steps of this tile of query rows so far
        uint32_t tile_count = 0;  // the CTA's steps before this segment
        segments([&](const Segment &seg) -> bool {
            const uint32_t first = tile_count;
            tile_count += seg.n;
            if (tile >= seg.tiles) return true;
            bool ok = true;
            // The queries: a warp copies its own 32 rows, consecutive lanes along a row.
            constexpr int kRowChunks = D / 8;
            const uint32_t q_to = sbase + tile * S::kQBytes;
            long long q_at = -1;  // of this lane's row
            {
                const int at = seg.q0 + tile * kPrefixRows + warp % 4 * 32 + lane, q_row = at / a.group;
                if (at < query_rows)
                    q_at = q_row * a.q_stride + static_cast<long long>(seg.head * a.group + at - q_row * a.group) * D;
            }
#pragma unroll 4
            for (int i = lane; i < 32 * kRowChunks; i += 32) {
                const int r = warp % 4 * 32 + i / kRowChunks, ch = i % kRowChunks;
                const long long from = __shfl_sync(0xFFFFFFFFu, q_at, i / kRowChunks);
                cp_async16_or_zeros(q_to + ch / 8 * S::kQChunkBytes + r * 128 + ((ch ^ r) & 7) * 16,
                                    a.q + (from < 0 ? 0 : from) + ch * 8, from >= 0);
            }
            cp_async_commit();
            cp_async_wait<0>();
            if (flip != 0u) {  // a negative scale: its own copies with the signs turned
                for (int i = lane; i < 32 * kRowChunks; i += 32) {
                    const int r = warp % 4 * 32 + i / kRowChunks, ch = i % kRowChunks;
                    uint4 *v = reinterpret_cast<uint4 *>(smem + tile * S::kQBytes + ch / 8 * S::kQChunkBytes + r * 128 +
                                                         ((ch ^ r) & 7) * 16);
                    *v = make_uint4(v->x ^ flip, v->y ^ flip, v->z ^ flip, v->w ^ flip);
                }
            }
            ptx::fence_proxy_async_shared();
            warp_arrive(bar_q + 8 * tile);

            float m = kNoMaximum, l = 0.0f;  // in units of log2
            for (int j = 0; j < seg.n; ++j, ++count) {
                if (!(ok = warp_wait(bar_s + 8 * tile, count & 1))) break;
                ptx::tc_fence_after_sync();
                uint32_t w[kTokens];
                ptx::tmem_ld_now(s_addr, w);
                ptx::tc_fence_before_sync();
                warp_arrive(bar_free + 8 * tile);
                const uint32_t *mask = masks + (first + j) % kMaskRing * S::kMaskWords;
                bool all = true;
#pragma unroll
                for (int i = 0; i < S::kMaskWords; ++i) all &= mask[i] == whole_mask(i);
                if (!all) {  // a NaN stays out of the maximum, and its weight is made 0 below
#pragma unroll
                    for (int e = 0; e < kTokens; ++e)
                        if (!(mask[e / 32] >> (e % 32) & 1)) w[e] = 0x7FC00000u;
                }
                float tops[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) tops[e] = __uint_as_float(w[e]);
#pragma unroll
                for (int e = 4; e + 1 < kTokens; e += 2)
                    tops[e / 2 & 3] = max3(tops[e / 2 & 3], __uint_as_float(w[e]), __uint_as_float(w[e + 1]));
                float top = fmaxf(max3(tops[0], tops[1], tops[2]), fmaxf(tops[3], -INFINITY));
                // -inf (no score, or only such) times 0 would be NaN.
                top = top == -INFINITY ? -INFINITY : top * c;
                // Every phase of bar_pv is waited for, in its turn.
                bool added = j == 0;
                if (__any_sync(0xFFFFFFFFu, top > m + 8.0f)) {
                    const float next = fmaxf(m, top), f = exp2_approx(m - next);
                    m = next;
                    l *= f;
                    if (j > 0) {
                        if (!(ok = warp_wait(bar_pv + 8 * tile, (count - 1) & 1))) break;
                        added = true;
                        ptx::tc_fence_after_sync();
#pragma unroll 1
                        for (int i = 0; i < D; i += 32) {
                            uint32_t o[32];
                            ptx::tmem_ld_now(o_addr + i, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            ptx::tmem_st_columns(o_addr + i, o);
                        }
                    }
                }
                float sum[4] = {};
                uint32_t p[kTokens / 2];
                auto weights = [&](auto masked) {
#pragma unroll
                    for (int e = 0; e < kTokens; e += 2) {
                        float x = __uint_as_float(w[e]), y = __uint_as_float(w[e + 1]);
                        fma2(x, y, c, -m);
                        x = exp2_approx(x);
                        y = exp2_approx(y);
                        if (masked) {
                            if (!(mask[e / 32] >> (e % 32) & 1)) x = 0.0f;
                            if (!(mask[e / 32] >> (e % 32) & 2)) y = 0.0f;
                        }
                        add2(sum[e & 2], sum[(e & 2) + 1], x, y);
                        p[e / 2] = pack_bf16(x, y);
                    }
                };
                if (all)
                    weights(std::false_type{});
                else
                    weights(std::true_type{});
                // The weights before are multiplied: waited for no sooner than here, so that the
                // way from one step's weights through their product to the next's is short.
                if (!added) {
                    if (!(ok = warp_wait(bar_pv + 8 * tile, (count - 1) & 1))) break;
                    ptx::tc_fence_after_sync();
                }
                ptx::tmem_st_columns(p_addr, p);
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                ptx::tmem_st_wait();
                ptx::tc_fence_before_sync();
                warp_arrive(bar_p + 8 * tile);
            }
            if (!ok || !warp_wait(bar_pv + 8 * tile, (count - 1) & 1)) return false;
            ptx::tc_fence_after_sync();
            // This segment's partial, 32 values of the warp's 32 rows at a time by way of its own rows
            // of the queries' first chunk (they are multiplied): a thread's own row would
            // go out in 16-byte pieces of 32 rows at once, 5700 clocks where this takes 1500.
            const int row0 = tile * kPrefixRows + warp % 4 * 32;
            float *slot = a.slots + (static_cast<size_t>(range + seg.head) * a.blocks + seg.block) * a.slot_floats;
            uint4 *stage = reinterpret_cast<uint4 *>(smem + tile * S::kQBytes + warp % 4 * 4096);
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                ptx::tmem_ld_now(o_addr + i, o);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    stage[lane * 8 + (e ^ (lane & 7))] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = e * 4 + lane / 8;
                    if (seg.q0 + row0 + r < query_rows)
                        __stcg(reinterpret_cast<uint4 *>(slot + static_cast<size_t>(row0 + r) * D + i) + lane % 8,
                               stage[r * 8 + ((lane ^ r) & 7)]);
                }
            }
            if (seg.q0 + row0 + lane < query_rows) {
                __stcg(slot + NT * kPrefixRows * D + row0 + lane, m);
                __stcg(slot + NT * kPrefixRows * (D + 1) + row0 + lane, l);
            }
            __syncwarp();  // the place is read: the next queries may come
            ptx::tc_fence_before_sync();  // O is read: before the next segment's arrival
            return true;
        });
    } else if (warp < S::kScoresWarp) {
        // ---------------- loaders ----------------
        ptx::give_registers<S::kOtherRegisters>();
        const int loader = (warp - S::kLoaderWarp) % S::kLoaders, kv = (warp - S::kLoaderWarp) / S::kLoaders;
        const uint16_t *from = kv == 0 ? a.k : a.v;
        const CUtensorMap *map = kv == 0 ? &k_map : &v_map;
        uint32_t *masks = reinterpret_cast<uint32_t *>(smem + S::kMaskOffset);
        constexpr int kRowChunks = D / 8, kRows = kTokens / S::kLoaders;  // cp.async: a warp's rows of a tile
        constexpr int kMine = (kRows + 31) / 32;                          // .. whose places a lane looks up
        static_assert(kTokens / 8 <= 32 && kTokens % (2 * S::kLoaders) == 0 && kRows * kRowChunks % 32 == 0, "whole rounds");
        int unit = kv;  // of the ring, so far
        uint32_t tile_count = 0;
        bool ok = true;
        auto publish = [&](int u) {  // this warp's part of a unit whose copies are complete
            ptx::fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_full + 8 * Ring::stage(u));
        };
        const int boxes = a.box_rows > 0 ? kTokens / a.box_rows : 0;
        const int items = S::kMerged ? boxes : boxes * S::kChunks;  // copies of a unit
        // This warp's bytes of a unit that comes by boxes.
        const int box_bytes = (items - loader + S::kLoaders - 1) / S::kLoaders * a.box_rows * 128 * (S::kMerged ? S::kChunks : 1);
        auto boxed = [&](int tile) { return boxes > 0 && (tile + 1) * kTokens <= length; };
        int head = 0, t = 0;  // of the tile that is looked up
        // Its places: lane's box (page and token within it), or the lane's row of this warp's.
        long long next[kMine];
        int next_page = 0, next_token = 0;
        auto look_up = [&]() {
            if (boxed(t)) {
                if (lane >= boxes) return;
                const int token = t * kTokens + lane * a.box_rows;
                const int e = a.page_shift >= 0 ? token >> a.page_shift : token / a.page_size;
                next_page = __ldcg(a.table + e);
                next_token = token - e * a.page_size;
            } else {
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    next[i] = i * 32 + lane < kRows ? place(head, t * kTokens + loader * kRows + i * 32 + lane) : -1;
            }
        };
        if (x_begin < x_end) {
            head = x_begin / steps;
            t = x_begin - head * steps;
            look_up();
        }
        const int first_head = head, first_t = t;
        for (int block = lane_block; ok && block < a.blocks; block += a.lanes) {
            for (int x = x_begin; ok && x < x_end; ++x, ++tile_count) {
                uint32_t *mask = masks + tile_count % kMaskRing * S::kMaskWords;
                const bool by_box = boxed(t);
                const int this_head = head, token = next_token;
                long long row_at[kMine];
#pragma unroll
                for (int i = 0; i < kMine; ++i) row_at[i] = next[i];
                int page = next_page;
                if (by_box) {
                    const bool there = lane >= boxes || (page >= 0 && page < a.num_pages);
                    const uint32_t good = __ballot_sync(0xFFFFFFFFu, there);
                    if (!there) {
                        atomicOr(&g_prefix_err, kErrRange);
                        page = a.num_pages;  // past the end: zeros
                    }
                    if (kv == 0 && loader == 0 && lane < S::kMaskWords) {
                        uint32_t bits = whole_mask(lane);
                        if (good != 0xFFFFFFFFu) {
                            bits = 0;
                            for (int e = 0; e < 32 && lane * 32 + e < kTokens; ++e)
                                bits |= (good >> ((lane * 32 + e) / a.box_rows) & 1u) << e;
                        }
                        mask[lane] = bits;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kMine; ++i)
                        if (i * 32 + lane < kRows && row_at[i] < 0 && t * kTokens + loader * kRows + i * 32 + lane < length)
                            atomicOr(&g_prefix_err, kErrRange);
                    if (kv == 0 && loader == 0) {
                        for (int i = 0; i < S::kMaskWords; ++i) {
                            const int at = i * 32 + lane;
                            const uint32_t bits = __ballot_sync(0xFFFFFFFFu, at < kTokens && place(head, t * kTokens + at) >= 0);
                            if (lane == 0) mask[i] = bits;
                        }
                    }
                }
                if (x + 1 == x_end) {  // the next block's first
                    head = first_head;
                    t = first_t;
                } else if (++t == steps) {
                    t = 0;
                    ++head;
                }
                if (x + 1 < x_end || block + a.lanes < a.blocks) look_up();
                const int s = Ring::stage(unit);
                const uint32_t to = sbase + S::kRingOffset + s * S::kUnitBytes;
                // The first round finds the stages free.
                if (!(ok = warp_wait(bar_empty + 8 * s, (Ring::round(unit) & 1) ^ 1))) break;
                if (by_box) {
                    __syncwarp();  // the mask is written
                    if (lane == 0) ptx::mbar_arrive_expect_tx(bar_full + 8 * s, box_bytes);
                    __syncwarp();
                    // The lanes' boxes come one after another.
                    const int item = loader + lane * S::kLoaders;
                    const int box = S::kMerged ? item : item / S::kChunks, ch = S::kMerged ? 0 : item % S::kChunks;
                    const int box_page = __shfl_sync(0xFFFFFFFFu, page, box & 31);
                    const int box_token = __shfl_sync(0xFFFFFFFFu, token, box & 31);
                    if (item < items) {
                        const uint32_t dst = to + ch * S::kChunkBytes + box * a.box_rows / 8 * S::kGroupBytes;
                        if constexpr (S::kMerged)
                            ptx::tma_load_5d(dst, map, bar_full + 8 * s, 0, 0, this_head * a.head_chunks, box_token / 8, box_page);
                        else
                            ptx::tma_load_4d(dst, map, bar_full + 8 * s, ch * 64, box_token, this_head, box_page);
                    }
                    unit += 2;
                    continue;
                }
#pragma unroll 4
                for (int i = 0; i < kRows * kRowChunks / 32; ++i) {
                    const int id = i * 32 + lane, own = id / kRowChunks, r = loader * kRows + own, ch = id % kRowChunks;
                    long long at = __shfl_sync(0xFFFFFFFFu, row_at[0], own & 31);
                    if constexpr (kMine > 1) {
                        const long long second = __shfl_sync(0xFFFFFFFFu, row_at[kMine - 1], own & 31);
                        if (own >= 32) at = second;
                    }
                    cp_async16_or_zeros(to + r / 8 * S::kGroupBytes + ch / 8 * S::kChunkBytes + r % 8 * 128 + ((ch ^ r) & 7) * 16,
                                        from + (at < 0 ? 0 : at) + ch * 8, at >= 0);
                }
                cp_async_commit();
                if (boxes > 0) {  // the tile that the prefix ends in
                    cp_async_wait<0>();
                    publish(unit);
                } else if (unit >= 2 * S::kLag) {
                    cp_async_wait<S::kLag>();
                    publish(unit - 2 * S::kLag);
                }
                unit += 2;
            }
        }
        if (lane == 0) tail[2 + warp - S::kLoaderWarp] = boxes > 0 ? unit : 0;  // the boxes begun
        cp_async_wait<0>();
        if (ok && boxes == 0)
            for (int u = max(kv, unit - 2 * S::kLag); u < unit; u += 2) publish(u);
    } else {
        ptx::give_registers<S::kOtherRegisters>();
    }
    auto full = [&](int u) {
        if (!wait(bar_full + 8 * Ring::stage(u), Ring::round(u) & 1)) return false;
        ptx::tc_fence_after_sync();
        return true;
    };
    // When every tile's products with a unit are complete it is free; a block's only tile speaks
    // for both.
    auto release = [&](int u, bool alone) {
        ptx::mma_commit(bar_empty + 8 * Ring::stage(u));
        if (NT == 2 && alone) ptx::mma_commit(bar_empty + 8 * Ring::stage(u));
    };
    // The issuers are one thread each: the waits and commits of one pass while another's products
    // run (a single issuer for all four took twice the time).
    if (warp >= S::kScoresWarp && warp < S::kValuesWarp && lane == 0) {
        // ---------------- MMA issuer: a tile's scores ----------------
        constexpr uint32_t idesc = ptx::idesc_bf16_f32(kPrefixRows, kTokens);
        const int tile = warp - S::kScoresWarp;
        const uint64_t q = ptx::smem_desc_sw128_kmajor(sbase + tile * S::kQBytes);
        int unit = 0;
        uint32_t scored = 0, loaded = 0;  // steps and segments
        segments([&](const Segment &seg) -> bool {
            if (tile >= seg.tiles) {
                unit += 2 * seg.n;
                return true;
            }
            if (!wait(bar_q + 8 * tile, loaded++ & 1)) return false;
            for (int j = 0; j < seg.n; ++j, ++scored, unit += 2) {
                // The step's before are read, and the keys are there.
                if (scored > 0 && !wait(bar_free + 8 * tile, (scored - 1) & 1)) return false;
                if (!full(unit)) return false;
                const uint64_t k =
                    ptx::smem_desc_sw128_kmajor(sbase + S::kRingOffset + Ring::stage(unit) * S::kUnitBytes, S::kGroupBytes);
#pragma unroll
                for (int s = 0; s < D / 16; ++s)  // addresses in the descriptors are in units of 16 bytes
                    ptx::mma_bf16(tmem + tile * kTokens, q + s / 4 * (S::kQChunkBytes / 16) + s % 4 * 2,
                                  k + s / 4 * (S::kChunkBytes / 16) + s % 4 * 2, idesc, s > 0);
                ptx::mma_commit(bar_s + 8 * tile);
                ptx::mbar_arrive(bar_s + 8 * tile);  // what the loader wrote before the keys, too
                release(unit, seg.tiles == 1);
            }
            return true;
        });
    } else if (warp >= S::kValuesWarp && warp < S::kValuesWarp + NT && lane == 0) {
        // ---------------- MMA issuer: a tile's output ----------------
        constexpr uint32_t idesc = ptx::idesc_bf16_f32(kPrefixRows, D) | ptx::kIdescBMnMajor;
        const int tile = warp - S::kValuesWarp;
        int unit = 1;
        uint32_t added = 0;
        // The self-test: nothing completes that barrier, so this wait runs out and ends every other.
        const bool ok = !a.selftest || tile > 0 || wait(bar_drain, 0);
        if (ok) segments([&](const Segment &seg) -> bool {
            if (tile >= seg.tiles) {
                unit += 2 * seg.n;
                return true;
            }
            for (int j = 0; j < seg.n; ++j, unit += 2) {
                if (!full(unit) || !wait(bar_p + 8 * tile, added++ & 1)) return false;
                ptx::tc_fence_after_sync();
                const uint64_t v = ptx::smem_desc_sw128_mnmajor(sbase + S::kRingOffset + Ring::stage(unit) * S::kUnitBytes,
                                                                S::kChunkBytes, S::kGroupBytes);
#pragma unroll
                for (int s = 0; s < kTokens / 16; ++s)
                    ptx::mma_bf16_tmem_a(tmem + S::kOCol + tile * D, tmem + S::kPCol + tile * (kTokens / 2) + s * 8,
                                         v + s * (S::kGroupBytes / 8), idesc, s > 0 || j > 0);
                ptx::mma_commit(bar_pv + 8 * tile);
                release(unit, seg.tiles == 1);
            }
            return true;
        });
    }
    __syncwarp();
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (*abort_flag) {
        // Nothing may still read or write this CTA's shared or tensor memory when it ends.
        auto drain = [&](uint32_t bar, uint32_t parity, uint64_t t0) {
            while (!ptx::mbar_try_wait(bar, parity))
                if (ptx::global_timer_ns() - t0 > kDrainLimitNs) {
                    atomicOr(&g_prefix_err, kErrLeft);
                    break;
                }
        };
        if (warp >= S::kScoresWarp && warp < S::kValuesWarp + NT && lane == 0) {
            ptx::mma_commit(bar_drain);
            drain(bar_drain, 0, ptx::global_timer_ns());
        }
        if (warp >= S::kLoaderWarp && warp < S::kScoresWarp && lane == 0) {
            // Units that the other loader of the kind has begun and this one has not lack this one's
            // arrival.
            const int mine = tail[2 + warp - S::kLoaderWarp], other = tail[2 + ((warp - S::kLoaderWarp) ^ 1)];
            const int end = max(mine, other);
            for (int u = mine; u < end; u += 2) ptx::mbar_arrive(bar_full + 8 * Ring::stage(u));
            const uint64_t t0 = ptx::global_timer_ns();
            for (int u = Ring::first_on_its_way(end); u < end; u += 2)
                drain(bar_full + 8 * Ring::stage(u), Ring::round(u) & 1, t0);
        }
        __syncthreads();
    }
    if (warp == S::kScoresWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, S::kTmemCols);
    }
}

// ---- the join ----
// One CTA for one head of one row: the prefix's partials of its query row, dealt to the warps,
// and the row's own tokens' result; then the warps' sums in order. All in L2, read once.
constexpr int kJoinWarps = 4;

// kAhead: parts whose loads a warp has on their way together.
template <int D, int kAhead>
__global__ void __launch_bounds__(kJoinWarps * 32) prefix_join_kernel(const PrefixArgs a) {
    constexpr int kValues = D / 32;
    __shared__ float sm_top[kJoinWarps], sm_weight[kJoinWarps], sm_o[kJoinWarps][D];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int job = blockIdx.x;
    ptx::pdl_launch_dependents();
    const int row = job / a.q_heads, h = job - row * a.q_heads;
    const int head = h / a.group, at = row * a.group + h - head * a.group;  // query row of the key head
    const int per = kPrefixRows * prefix_tiles(D, static_cast<long long>(a.rows) * a.group);
    const int block = at / per, in_block = at - block * per;
    ptx::pdl_wait();
    const int length = min(max(__ldcg(a.length), 0), a.capacity);
    const int steps = (length + a.tokens - 1) / a.tokens;
    const PrefixCut cut(steps * a.kv_heads, a.ranges);
    const int first = steps > 0 ? cut.owner(head * steps) : 0;
    const int parts = steps > 0 ? cut.owner(head * steps + steps - 1) - first + 1 : 0;
    const float *slots = a.slots + (static_cast<size_t>(first + head) * a.blocks + block) * a.slot_floats;
    const size_t stride = static_cast<size_t>(a.blocks) * a.slot_floats;  // from part to part
    const float *maxima = slots + static_cast<size_t>(per) * D + in_block, *sums = maxima + per;
    const float *values = slots + static_cast<size_t>(in_block) * D + lane;

    // This warp's parts; the first warp begins with the row's own tokens (sum of weights 2^own).
    float o[kValues], top = kNoMaximum, weight = 0.0f;
#pragma unroll
    for (int e = 0; e < kValues; ++e) o[e] = 0.0f;
    if (warp == 0) {
        const float own = __ldcg(a.own_lse + job) * kLog2e;
        if (own != -INFINITY) {
            top = fmaxf(own, kNoMaximum);
            weight = exp2_approx(own - top);
#pragma unroll
            for (int e = 0; e < kValues; ++e)
                o[e] = weight * __ldcg(a.own_out + static_cast<size_t>(job) * D + lane + e * 32);
        }
    }
    for (int s0 = warp; s0 < parts; s0 += kAhead * kJoinWarps) {
        float m[kAhead], l[kAhead], v[kAhead][kValues], next = top;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const size_t s = s0 + u * kJoinWarps;
            const bool there = s < static_cast<size_t>(parts);
            m[u] = there ? __ldcg(maxima + s * stride) : kNoMaximum;
            l[u] = there ? __ldcg(sums + s * stride) : 0.0f;
#pragma unroll
            for (int e = 0; e < kValues; ++e) v[u][e] = there ? __ldcg(values + s * stride + e * 32) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) next = fmaxf(next, m[u]);
        const float f = exp2_approx(top - next);
        top = next;
        weight *= f;
#pragma unroll
        for (int e = 0; e < kValues; ++e) o[e] *= f;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float w = exp2_approx(m[u] - top);
            weight += w * l[u];
#pragma unroll
            for (int e = 0; e < kValues; ++e) o[e] += w * v[u][e];
        }
    }
    if (lane == 0) sm_top[warp] = top, sm_weight[warp] = weight;
#pragma unroll
    for (int e = 0; e < kValues; ++e) sm_o[warp][lane + e * 32] = o[e];
    __syncthreads();
    float all = sm_top[0], sum = 0.0f, f[kJoinWarps];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) all = fmaxf(all, sm_top[w]);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        f[w] = exp2_approx(sm_top[w] - all);
        sum += f[w] * sm_weight[w];
    }
    const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
    for (int i = threadIdx.x; i < D; i += kJoinWarps * 32) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) v += f[w] * sm_o[w][i];
        a.out[static_cast<size_t>(job) * D + i] = __bfloat16_as_ushort(__float2bfloat16_rn(v * inv));
    }
    if (a.lse != nullptr && threadIdx.x == 0)
        a.lse[job] = sum > 0.0f || sum != sum ? (all + log2f(sum)) * kLn2 : -INFINITY;
}

template <int D, int NT>
cudaError_t launch_prefix(const CUtensorMap &k_map, const CUtensorMap &v_map, const PrefixArgs &a,
                          int device, cudaStream_t stream, bool pdl) {
    using S = Shape<D, NT>;
    static bool configured[64] = {};
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    if (!configured[device]) {
        cudaError_t e = cudaFuncSetAttribute(prefix_attention_kernel<D, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::kDynamicBytes);
        if (e != cudaSuccess) return e;
        // The softmax warps' registers come out of what the block is launched with: with fewer they
        // would wait for them forever.
        cudaFuncAttributes f;
        if ((e = cudaFuncGetAttributes(&f, prefix_attention_kernel<D, NT>)) != cudaSuccess) return e;
        if (f.numRegs < S::kLaunchRegisters) return cudaErrorInvalidConfiguration;
        configured[device] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ranges * a.lanes, 1, 1);
    cfg.blockDim = dim3(S::kThreads, 1, 1);
    cfg.dynamicSmemBytes = S::kDynamicBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, prefix_attention_kernel<D, NT>, k_map, v_map, a);
}

template <int D, int kAhead>
cudaError_t launch_join_kernel(const PrefixArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * a.q_heads, 1, 1);
    cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;  // behind the library's own kernels
    return cudaLaunchKernelEx(&cfg, prefix_join_kernel<D, kAhead>, a);
}

// 8 parts a warp while all CTAs run at once (four an SM), 4 and more CTAs an SM beyond: 64 rows x 7
// heads behind 16001 tokens 22.5 us in all with 8, 23.1 with 4; 64 x 56 over 8 behind 8000 52.1 and
// 45.3, behind 65521 157.5 and 150.8; 64 x 32 over 4 of 64 behind 16001 38.9 and 35.0. Always 4 for
// wide heads, a part of which is as many registers.
template <int D>
cudaError_t launch_join(const PrefixArgs &a, int num_sms, cudaStream_t stream) {
    if constexpr (D <= 128)
        if (static_cast<long long>(a.rows) * a.q_heads <= 4ll * num_sms) return launch_join_kernel<D, 8>(a, stream);
    return launch_join_kernel<D, 4>(a, stream);
}

}  // namespace

int prefix_box_rows(int page_size, int tokens) {
    const int both = page_size | tokens, rows = both & -both;  // the largest power of two that divides both
    return rows >= 8 ? rows : 0;
}

cudaError_t launch_prefix_attention(const CUtensorMap &k_map, const CUtensorMap &v_map, const PrefixArgs &a,
                                    int head_dim, int device, cudaStream_t stream, bool pdl) {
    const bool two = prefix_tiles(head_dim, static_cast<long long>(a.rows) * a.group) == 2;
    switch (head_dim) {
        case 64:
            if (two) return launch_prefix<64, 2>(k_map, v_map, a, device, stream, pdl);
            return launch_prefix<64, 1>(k_map, v_map, a, device, stream, pdl);
        case 96:
            if (two) return launch_prefix<96, 2>(k_map, v_map, a, device, stream, pdl);
            return launch_prefix<96, 1>(k_map, v_map, a, device, stream, pdl);
        case 128:
            if (two) return launch_prefix<128, 2>(k_map, v_map, a, device, stream, pdl);
            return launch_prefix<128, 1>(k_map, v_map, a, device, stream, pdl);
        case 192: return launch_prefix<192, 1>(k_map, v_map, a, device, stream, pdl);
        case 256: return launch_prefix<256, 1>(k_map, v_map, a, device, stream, pdl);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_prefix_join(const PrefixArgs &a, int head_dim, int num_sms, cudaStream_t stream) {
    switch (head_dim) {
        case 64: return launch_join<64>(a, num_sms, stream);
        case 96: return launch_join<96>(a, num_sms, stream);
        case 128: return launch_join<128>(a, num_sms, stream);
        case 192: return launch_join<192>(a, num_sms, stream);
        case 256: return launch_join<256>(a, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t prefix_error_word(int **word) { return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_prefix_err); }

}  // namespace skinny

