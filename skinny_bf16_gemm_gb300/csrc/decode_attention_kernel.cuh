// Attention of one new token per row over a paged key-value cache on GB300 (sm_103a).
//
//   s_j = scale q.k_j,  m = max s_j,  l = sum exp(s_j - m),  o = sum exp(s_j - m) v_j / l
// over the tokens j the row sees: all before its length, or with a sliding window
// the last `window` of them and the first `sinks`. One pass over the cache with the
// running maximum and sum; the query heads that share a key head are done together,
// so every key and value is read once. Bound by HBM: 4 D bytes a token and key head
// against 4 G D flops (G heads sharing) -- 8 flops a byte for G = 8.
//
// CTAs of 4 warps, one or two to an SM; every warp has an equal share of the tiles
// (attention_plan.cuh), streams it through a private ring of cp.async stages and keeps
// its own maximum, sum and accumulator, so nothing in the main loop waits for another
// warp. The ring runs across items. It is filled by 16-byte copies with each token's
// address from the block table, so pages of any size, tokens at any 16-byte-aligned
// strides and ranges that end inside a page are all the same to it. A copy engine's
// tensor loads would want pages of a multiple of the tile; one bulk copy per row was not
// tried.
// The products run on the tensor cores with tokens (scores) and head dimension (output)
// as the 16 rows of mma.sync and the query heads as its 8 columns. HBM feeds an SM 23
// bytes a clock, 8 KB (16 tokens of 128) in 356 clocks; the 24 MMAs of those tokens take
// 48 clocks of its four tensor cores (1024 multiply-adds a clock, measured), so a larger
// MMA's set-up through tensor memory would buy nothing for one block of 8 heads. With 32
// heads to a key head the instructions around the MMAs are the bound (see below).
// Weights p are split into two BF16 terms (p truncated, and the rest rounded: within
// 2^-15 of p), so the product with V loses nothing that the BF16 output shows; maxima
// and sums are FP32.
//
// An item that is one warp's alone is stored from its registers. Other warps' partials
// are joined by the CTA through shared memory, and an item whose tiles span several CTAs
// by whichever of them is last to publish its part (a counter in the workspace): it adds
// the parts in order, so the bits do not depend on who was last. More than 20 parts are
// joined in two such levels, in about as many groups as a group has parts, to keep the last
// reader's share short. No CTA waits for another.
//
// Measured on GB300 (graph of calls; bytes of keys and values over the time): 131071
// tokens of 8 key heads of 128, 56 query heads, 88 us, 6.1 TB/s; 64 ragged rows to 16384
// of 8 x 64 163-187 us (the two layouts), 5.6-6.4 TB/s; a window of 4096 in 32 rows 82 us,
// 5.8 TB/s; 64 ragged rows to 4000 of one key head 20 us; one row of 129 tokens 7.2 us.
// What is left over the floor: about 1.5 us until the lengths' prefix sums and shares are
// known and 1.5 us to the first tile; SMs that get less of the memory's bandwidth than the
// average (their CTAs end last); the joins, 3 us for one level and 3 us more for a second;
// from 16 heads to a key head on, and at 192 and 256, the chain of instructions of a step.
// Tried and not faster: keys refilled before the softmax (the copies' issue waits for the
// memory system, and the softmax with it), 8 warps a CTA, two CTAs an SM of 128-wide heads
// with one set of 16 tokens a step (131071 tokens 92-96 us; 64 rows to 4000 18.3), L2
// prefetch sizes on the copies, chunks dealt out as CTAs come free (each costs a join),
// several items of a CTA joined by a warp or two each (3 % slower for one row of one item).
//
// Two more forms serve decode_attention_shared_prefix_bf16. kPart: the rows' own tokens of a batch
// behind a shared prefix; the result stays FP32, for the join with the prefix
// (prefix_attention.cu). That kernel may run beside this one, which waits for it only at its
// end, so that whatever waits for this kernel has waited for both. kJoined: the prefix's
// tokens come before every row's own, from a table of their own.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "attention_plan.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace skinny {
namespace {

// The maximum of no scores: finite, so that exp2(-inf - m) is 0 and exp2(m - m) is 1.
constexpr float kNoMaximum = -3.402823466e+38f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kWarps = kAttnWarps;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxGroups = 32;   // groups of the second level of a join
constexpr int kSnapShare = 2;    // items of so many tiles are not cut by warps' shares
__device__ int g_attn_err;  // nonzero: a length or page index was out of range

template <int D, int NB>
struct Shape {
    // A tile is a warp's step: 16 tokens, or two such sets side by side, whose chains of
    // dependent instructions overlap, where registers and rings allow (16 rows to 8192 of
    // 128-wide heads 39.5 us, 42.4 with one set, three stages and two CTAs an SM; of 192-wide,
    // whose two sets' copies queue too long, 36.9 us with two and 34.6 with one).
    static constexpr int kSets = NB == 1 && D <= 128 ? 2 : 1;
    static constexpr int kSub = 16 * kSets;
    static constexpr int kRowBytes = D * 2;
    static constexpr int kStageBytes = 2 * kSub * kRowBytes;  // keys, then values
    // One stage is read while the other's copies are on their way: 64 KB an SM for 64-, 128-
    // and 256-wide heads. A third is slower everywhere (131071 tokens of 128: 90 us, 95 with
    // three; 16 heads to a key head 46 and 50; 256-wide 37 and 43): with more of every SM's
    // copies queued the SMs that get less of the memory's bandwidth fall further behind.
    static constexpr int kStages = 2;
    static constexpr int kSlots = kStages + 1;  // lookups on their way
    static constexpr int kHeads = 8 * NB;
    static constexpr int kSlotFloats = attn_slot_floats(D, NB);
    static constexpr int kRingBytes = std::max(kStages * kStageBytes, kSlotFloats * 4);  // per warp
    static constexpr int kMaximaAt = kHeads * D;  // in a partial: the maxima, then the sums
    // A warp's last partial is kept in its ring, which is empty by then; one of an item
    // that ends earlier in its share here, if there is room, else in the workspace.
    static constexpr bool kEarlyShared = kWarps * (kRingBytes + kSlotFloats * 4) <= 216 * 1024 / attn_ctas_per_sm(D, NB);
    static constexpr int kEarlyOffset = kWarps * kRingBytes;
    static constexpr int kFactorOffset = kEarlyOffset + (kEarlyShared ? kWarps * kSlotFloats * 4 : 0);
    static constexpr int kMlOffset = kFactorOffset + kMaxGroups * kHeads * 4;  // factors [kMaxGroups][kHeads]
    static constexpr int kLookOffset = kMlOffset + 2 * kHeads * 4;             // m, l of a join
    static constexpr int kRowsOffset = kLookOffset + kWarps * kSlots * (kSub + 1) * 8;  // prefix, lengths
    static_assert(kRingBytes % 16 == 0, "16-byte copies");
    static_assert(kSub >= kAttnMinTile, "the host counts tiles of kAttnMinTile");
    static_assert(kLookOffset % 8 == 0, "64-bit places");
    static_assert(kRowsOffset + (2 * kAttnMaxRows + 1) * 4 + 3 * 1024 <= 232448, "with the static arrays");
    static int bytes(int rows) { return kRowsOffset + (2 * rows + 1) * 4; }
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zeros(uint32_t dst, const void *src, bool full) {
    const int bytes = full ? 16 : 0;  // 0: the 16 bytes are zero-filled, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
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

// What truncating a weight p >= 0 to BF16 leaves, of a weight above 0 at least BF16's
// smallest value: both its terms are then positive, so that an infinite value comes out
// infinite and not 0 * inf or inf - inf. That is under 2^-15 of any weight from 2^-118 on. A
// weight that underflowed, to 0 below 2^-126, adds nothing of a finite value. (One more
// minimum a weight: 32 heads of 128 to a key head 67.4 us, 66.9 without; else no difference.)
__device__ __forceinline__ float rest_of(float p) {
    return fmaxf(p - __uint_as_float(__float_as_uint(p) & 0xFFFF0000u), fminf(p, 9.18354962e-41f));
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

// x / d for 0 <= x < 2^31, d > 0 and a quotient below 2^20: the float quotient is off by
// less than one, which the remainder's sign shows. A third of an integer division's time.
__device__ __forceinline__ int quotient(int x, int d) {
    const int q = static_cast<int>(__fdividef(static_cast<float>(x), static_cast<float>(d)));
    const int r = static_cast<int>(static_cast<unsigned>(x) - static_cast<unsigned>(q) * static_cast<unsigned>(d));
    return r < 0 ? q - 1 : r >= d ? q + 1 : q;
}

// An even cut of `tiles` tiles into `parts` (at most 2^20): the first `extra` parts have
// base + 1.
struct Cut {
    int base, extra;
    __device__ Cut(int tiles, int parts) {
        base = tiles / parts;
        extra = tiles - base * parts;
    }
    __device__ int begin(int c) const { return c * base + min(c, extra); }
    __device__ int owner(int x) const {
        const int at = extra * (base + 1);
        const bool low = x < at;
        return (low ? 0 : extra) + quotient(low ? x : x - at, low ? base + 1 : base);
    }
};

enum Form { kWhole, kPart, kJoined };
template <int FORM>
using ArgsOf = std::conditional_t<FORM == kWhole, AttentionArgs, SharedAttentionArgs>;

// kPart: what the kernel's end, wherever it is, waits for.
struct WaitAtTheEnd {
    __device__ __forceinline__ ~WaitAtTheEnd() { ptx::pdl_wait(); }
};
struct NoWait {};

template <int D, int NB, int FORM>
__global__ void __launch_bounds__(kThreads, attn_ctas_per_sm(D, NB)) decode_attention_kernel(const ArgsOf<FORM> a) {
    using S = Shape<D, NB>;
    constexpr bool PART = FORM == kPart, JOINED = FORM == kJoined;
    [[maybe_unused]] const std::conditional_t<PART, WaitAtTheEnd, NoWait> end;
    constexpr int kSub = S::kSub, kSets = S::kSets, kSlots = S::kSlots;
    constexpr uint32_t kAllSeen = kSub == 32 ? 0xFFFFFFFFu : (1u << (kSub & 31)) - 1u;
    constexpr int kChunks = D / 8;            // 16-byte chunks of a token's row
    constexpr int kCopies = kSub * kChunks / 32;
    constexpr int kSteps = D / 16;
    // Chunk c of token row r is kept at chunk c ^ swizzle(r): eight rows of one chunk
    // then cover all banks. Rows of 96 values alternate between the two halves of the
    // banks by themselves, so two bits are enough (and all that 12 chunks allow).
    constexpr bool kWide = kChunks % 8 == 0;
    auto swizzle = [](int r) { return kWide ? r & 7 : (r >> 1) & 3; };
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint4 sm_q[kWarps][32];
    __shared__ uint32_t sm_valid[kWarps][S::kStages];
    __shared__ uint32_t sm_places[kWarps][kSub];
    __shared__ int sm_scan[kWarps];
    __shared__ int sm_key[2 * kWarps];  // items of the warps' partials, -1: none
    __shared__ int sm_last[3];  // arrivals that were the last: two items' chunks, a group
    const uint32_t sbase = ptx::smem_addr(smem);
    int *prefix = reinterpret_cast<int *>(smem + S::kRowsOffset);
    int *lengths = prefix + a.rows + 1;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int cta = blockIdx.x;

    ptx::pdl_launch_dependents();
    if (!PART) ptx::pdl_wait();

    // ---- the split ----
    int shared = 0;  // JOINED: tokens of the prefix
    if constexpr (JOINED) {
        shared = __ldcg(a.prefix_length);
        if (shared < 0 || shared > a.prefix_capacity) {
            if (cta == 0 && tid == 0) atomicOr(&g_attn_err, 1);
            shared = shared < 0 ? 0 : a.prefix_capacity;
        }
    }
    // Prefix sums of the rows' tiles. A length is taken within [0, capacity].
    const int per = (a.rows + kThreads - 1) / kThreads;
    const int r_lo = min(tid * per, a.rows), r_hi = min(r_lo + per, a.rows);
    int mine = 0;
    for (int r = r_lo; r < r_hi; ++r) {
        int n = __ldcg(a.lengths + r);
        if (n < 0 || n > a.capacity) {
            if (cta == 0) atomicOr(&g_attn_err, 1);
            n = n < 0 ? 0 : a.capacity;
        }
        if constexpr (JOINED) n += shared;
        lengths[r] = n;
        mine += (seen_of(n, a.window, a.sinks).count + kSub - 1) / kSub;
        prefix[r + 1] = mine;
    }
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) sm_scan[warp] = scan;
    if (tid < 2 * kWarps) sm_key[tid] = -1;
    __syncthreads();
    int before = scan - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) before += sm_scan[w];
    for (int r = r_lo; r < r_hi; ++r) prefix[r + 1] += before;
    if (tid == 0) prefix[0] = 0;
    __syncthreads();

    // Rows that see nothing: zeros, and a log-sum of -inf.
    for (int r = cta; r < a.rows; r += gridDim.x) {
        if (prefix[r + 1] != prefix[r]) continue;
        if constexpr (!PART) {  // PART: a log-sum of -inf says enough
            uint4 *o = reinterpret_cast<uint4 *>(a.out + static_cast<size_t>(r) * a.q_heads * D);
            for (int i = tid; i < a.q_heads * kChunks; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
        }
        if (a.lse != nullptr)
            for (int h = tid; h < a.q_heads; h += kThreads)
                a.lse[static_cast<size_t>(r) * a.q_heads + h] = -INFINITY;
    }

    const int items_per_row = a.kv_heads * a.head_blocks;
    const int total = prefix[a.rows] * items_per_row;  // below 2^31 (host check)
    if (total == 0) return;
    // No fewer tiles a warp than `least`: one where items are short (64 rows to 200 tokens:
    // 8.4 us with one, 11.2 with two), two where every further piece makes a join longer
    // (4 rows to 9000: 14.1 us with two, 15.3 with one).
    const int least = quotient(total, a.rows * items_per_row) <= 32 ? 1 : 2;
    const int chunks = min(static_cast<int>(gridDim.x), (total + kWarps * least - 1) / (kWarps * least));
    if (cta >= chunks) return;
    const Cut cut(total, chunks);
    // Chunks do not cut items of up to `uncut` tiles: a few tiles more or less cost less than
    // a join over CTAs (32 rows of 8 heads to 1000 tokens: 20.6 us with 16, 22.4 with 8; one
    // row of 8 heads of 500 tokens, in chunks of 4 to 8 tiles: 9.3 with 8, 10.0 with 16).
    const int uncut = cut.base >= 8 ? 16 : 8;

    // A place in the tile sequence: tile `tile` of item `item` (key head and head block)
    // of row `row`.
    struct Place {
        int row, item, tile;
    };
    auto next_item = [&](Place &p) {  // only where a further tile exists
        p.tile = 0;
        if (++p.item == items_per_row) {
            p.item = 0;
            do ++p.row; while (prefix[p.row + 1] == prefix[p.row]);
        }
    };
    // The places of two tiles (the same two in the whole warp).
    auto find = [&](int x0, int x1, Place (&p)[2]) {
        const int xs[2] = {x0, x1};
        int at[2] = {-1, -1};  // rows: the first that ends after the tile
        for (int r0 = 0; at[0] < 0 || at[1] < 0; r0 += 32) {
            const int end = r0 + lane < a.rows ? prefix[r0 + lane + 1] * items_per_row : 0x7FFFFFFF;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned over = __ballot_sync(0xFFFFFFFFu, end > xs[i]);
                if (at[i] < 0 && over != 0) at[i] = r0 + __ffs(over) - 1;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int begin = prefix[at[i]], tiles = prefix[at[i] + 1] - begin;
            const int in_row = xs[i] - begin * items_per_row;
            const int item = quotient(in_row, tiles);
            p[i] = {at[i], item, in_row - item * tiles};
        }
    };
    // The end of a chunk or share that would be at tile x, at place p: not within an item of
    // at most `most` tiles.
    auto snap = [&](int x, Place &p, int most) -> int {
        const int tiles = prefix[p.row + 1] - prefix[p.row];
        if (p.tile == 0 || tiles > most) return x;
        const bool up = 2 * p.tile >= tiles;
        x += up ? tiles - p.tile : -p.tile;
        p.tile = 0;
        if (up && x < total) next_item(p);
        return x;
    };
    // This warp's share [x, x_end), and the place it begins at. The end of the sequence,
    // where there is no tile, stands for itself.
    int x, x_end;
    Place here;
    {
        const int last = total - 1;
        Place p[2];
        int b = cut.begin(cta), e = cut.begin(cta + 1);
        find(b, min(e, last), p);
        b = snap(b, p[0], uncut);
        if (e < total) e = snap(e, p[1], uncut);
        x = b + (e - b) * warp / kWarps;
        x_end = b + (e - b) * (warp + 1) / kWarps;
        find(min(x, last), min(x_end, last), p);
        if (x < total && warp > 0) x = snap(x, p[0], kSnapShare);
        if (x_end < total && warp < kWarps - 1) x_end = snap(x_end, p[1], kSnapShare);
        here = p[0];
    }

    // ---- the copies: one stage a tile ----
    // A stage is refilled as soon as it is read, so that while a warp waits its whole ring
    // is in flight. Lane t < kSub finds token t's address. Its page index comes by cp.async
    // too, kStages steps before the copy that needs it and in the group that is waited for
    // by then, so the block table's latency is hidden as the data's is (a lookup one step
    // ahead, which waited a full L2 trip every step, cost up to a third of the bandwidth).
    const uint32_t ring = sbase + warp * S::kRingBytes;
    long long *look_head = reinterpret_cast<long long *>(smem + S::kLookOffset) + warp * kSlots;
    int2 *look = reinterpret_cast<int2 *>(smem + S::kLookOffset + kWarps * kSlots * 8) + warp * kSlots * kSub;
    Place ahead = here;
    int ahead_x = x, ahead_tiles = 0;
    Seen ahead_seen = {};
    const int *ahead_table = nullptr;
    long long ahead_head = 0;
    auto enter = [&]() {  // `ahead` is at a new item
        ahead_tiles = prefix[ahead.row + 1] - prefix[ahead.row];
        ahead_seen = seen_of(lengths[ahead.row], a.window, a.sinks);
        ahead_table = a.block_table + ahead.row * a.table_stride;
        ahead_head = quotient(ahead.item, a.head_blocks) * a.head_stride;
    };
    if (x < x_end) enter();
    // Look the next tile up: this lane's token's place within its page (-1: none), and on
    // its way the page.
    auto look_up = [&](int slot) {
        int2 *to = look + slot * kSub + lane;
        int in_page = -1;
        if (ahead_x < x_end) {
            const int t = ahead.tile * kSub + lane;
            if (lane < kSub && t < ahead_seen.count) {
                int j = t < ahead_seen.sinks ? t : t + ahead_seen.gap;
                const bool own = !JOINED || j >= shared;
                if constexpr (JOINED) j -= own ? shared : 0;
                const int e = a.page_shift >= 0 ? j >> a.page_shift : j / a.page_size;
                in_page = j - e * a.page_size;
                if constexpr (JOINED)
                    cp_async4(ptx::smem_addr(&to->y), (own ? ahead_table : a.prefix_table) + e);
                else
                    cp_async4(ptx::smem_addr(&to->y), ahead_table + e);
            }
            if (lane == 0) look_head[slot] = ahead_head;
            if (++ahead.tile == ahead_tiles && ahead_x + 1 < x_end) {
                next_item(ahead);
                enter();
            }
            ++ahead_x;
        }
        if (lane < kSub) to->x = in_page;
    };
    // Fill a stage with the tile of a lookup slot. With every token there and 16-byte chunk
    // numbers of 32 bits, a row's place is one multiply-add away (the places go through
    // shared memory rather than shuffles, and rows are named by the few swizzles that occur,
    // so that the addresses need few registers); rows that are not there are zero-filled.
    uint32_t *places = sm_places[warp];
    auto fill = [&](int stage, int slot) {
        const int2 at = look[slot * kSub + (lane & (kSub - 1))];
        long long off = -1;
        if (lane < kSub && at.x >= 0) {
            if (at.y >= 0 && at.y < a.num_pages)
                off = at.y * a.page_stride + at.x * a.token_stride + look_head[slot];
            else
                atomicOr(&g_attn_err, 1);
        }
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, off >= 0);
        if (lane == 0) sm_valid[warp][stage] = valid;
        const uint32_t to = ring + stage * S::kStageBytes;
        auto share = [&]() {
            if (lane < kSub) places[lane] = off < 0 ? 0u : static_cast<uint32_t>(off >> 3);
            __syncwarp();
        };
        if (valid == kAllSeen && !a.wide) {
            share();
#pragma unroll
            for (int it = 0; it < kCopies; ++it) {
                int tok, ch, swz;
                if constexpr (32 % kChunks == 0) {
                    constexpr int kRows = 32 / kChunks;  // rows of one copy
                    tok = it * kRows + lane / kChunks;
                    ch = lane % kChunks;
                    swz = (lane / kChunks + it % (8 / kRows) * kRows) & 7;
                } else {
                    tok = (it * 32 + lane) / kChunks;
                    ch = (it * 32 + lane) % kChunks;
                    swz = swizzle(tok);
                }
                const size_t e = static_cast<size_t>(places[tok]) * 16;
                const uint32_t dst = to + (ch ^ swz) * 16 + tok * S::kRowBytes;
                cp_async16(dst, reinterpret_cast<const uint8_t *>(a.k + ch * 8) + e);
                cp_async16(dst + kSub * S::kRowBytes, reinterpret_cast<const uint8_t *>(a.v + ch * 8) + e);
            }
        } else if (valid != 0) {  // the last tile of an item, as a rule
            if (kSets == 2) share();
#pragma unroll(kSets == 2 ? 4 : 1)
            for (int it = 0; it < kCopies; ++it) {
                const int id = it * 32 + lane, tok = id / kChunks, ch = id % kChunks;
                const bool there = valid >> tok & 1;
                size_t e = kSets == 2 ? static_cast<size_t>(places[tok]) * 16 : 0;
                if (kSets == 1 || a.wide) {
                    const long long o = __shfl_sync(0xFFFFFFFFu, off, tok);
                    e = o < 0 ? 0 : static_cast<size_t>(o) * 2;
                }
                const uint32_t dst = to + tok * S::kRowBytes + (ch ^ swizzle(tok)) * 16;
                cp_async16_or_zeros(dst, reinterpret_cast<const uint8_t *>(a.k + ch * 8) + e, there);
                cp_async16_or_zeros(dst + kSub * S::kRowBytes, reinterpret_cast<const uint8_t *>(a.v + ch * 8) + e, there);
            }
        }
    };
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) look_up(i);
    cp_async_commit();

    // Queries as the MMA's B: head lane / 4 of each block of 8, values 2 (lane % 4) on.
    // 16-byte loads, then the fragments by way of 512 bytes of shared memory: loads of a
    // fragment each, 4 bytes a lane, kept one row's CTAs waiting for the L2 slices that hold
    // its queries (131071 tokens of one key head: 22.8 us, 19.1 this way). They are on their
    // way from the item before's last scores on where there are registers for them (16 rows to
    // 8192, 16 heads of 128 to a key head: 43.4 us, 45.1 without; 32 heads: 67 us without, which
    // spills 180 bytes, and 98 with them).
    constexpr bool kQueriesAhead = D * NB <= 256;
    uint32_t qf[kSteps][NB][2];
    uint4 qw[NB][kChunks / 4];
    auto load_queries = [&](const Place &p) {
        const int kv_head = quotient(p.item, a.head_blocks);
        const int g0 = (p.item - kv_head * a.head_blocks) * a.block_heads;
        const int n = min(a.block_heads, a.group - g0);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int h = b * 8 + lane / 4;
            const uint4 *q = reinterpret_cast<const uint4 *>(
                a.q + p.row * a.q_stride + static_cast<long long>(kv_head * a.group + g0 + h) * D) + (lane & 3);
#pragma unroll
            for (int i = 0; i < kChunks / 4; ++i) qw[b][i] = h < n ? __ldcg(q + i * 4) : make_uint4(0, 0, 0, 0);
        }
    };
    auto place_queries = [&]() {
        const int put = (lane & ~3) | ((lane ^ (lane >> 3)) & 3);
        const uint32_t get = ptx::smem_addr(sm_q[warp]) +
                             (((lane & 7) * 4 + (((lane >> 3) ^ ((lane & 7) >> 1)) & 3)) << 4);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < kChunks / 4; ++i) {
                sm_q[warp][put] = qw[b][i];
                __syncwarp();
                uint32_t r[4];
                ldmatrix4(r, get);
                __syncwarp();
                qf[2 * i][b][0] = r[0];
                qf[2 * i][b][1] = r[1];
                qf[2 * i + 1][b][0] = r[2];
                qf[2 * i + 1][b][1] = r[3];
            }
    };
    if (kQueriesAhead && x < x_end) load_queries(here);
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) {  // tile i is in lookup slot i mod kSlots
        fill(i, i);
        look_up(i == 0 ? S::kStages : i - 1);
        cp_async_commit();
        __syncwarp();
    }

    // An item's first output head, and how many it has.
    struct Heads {
        size_t first;
        int count;
    };
    auto heads_of = [&](int row, int item) -> Heads {
        const int kv_head = quotient(item, a.head_blocks);
        const int g0 = (item - kv_head * a.head_blocks) * a.block_heads;
        return {static_cast<size_t>(row) * a.q_heads + kv_head * a.group + g0, min(a.block_heads, a.group - g0)};
    };
    // A fragment of the output (16 values of 8 heads) from sums and the heads' 1 / l. The
    // transpose puts a head's values side by side in a lane.
    auto store_out = [&](const Heads &h, int s, int b, float v0, float v1, float v2, float v3, float inv0, float inv1) {
        if constexpr (PART) {  // values s * 16 + lane / 4 and + 8 of heads 2 (lane % 4) and + 1
            float *o = a.part + (h.first + b * 8 + (lane & 3) * 2) * D + s * 16 + lane / 4;
            if (b * 8 + (lane & 3) * 2 < h.count) o[0] = v0 * inv0, o[8] = v2 * inv0;
            if (b * 8 + (lane & 3) * 2 + 1 < h.count) o[D] = v1 * inv1, o[D + 8] = v3 * inv1;
            return;
        }
        const uint32_t w0 = movmatrix_trans(pack_bf16(v0 * inv0, v1 * inv1));
        const uint32_t w1 = movmatrix_trans(pack_bf16(v2 * inv0, v3 * inv1));
        if (b * 8 + lane / 4 < h.count) {
            uint32_t *o = reinterpret_cast<uint32_t *>(a.out + (h.first + b * 8 + lane / 4) * D + s * 16 + (lane & 3) * 2);
            o[0] = w0;
            o[4] = w1;
        }
    };
    auto store_lse = [&](const Heads &h, int at, float m, float l) {
        if (a.lse != nullptr && at < h.count)
            a.lse[h.first + at] = l > 0.0f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
    };
    auto inverse = [](float l) { return l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l); };
    auto slot_at = [&](int slot) { return a.partials + static_cast<size_t>(slot) * S::kSlotFloats; };
    // Partial e of this CTA's warps: 2 w of an item that ends within warp w's share, 2 w + 1
    // the last of the share.
    auto entry_at = [&](int e) -> float * {
        if (e & 1) return reinterpret_cast<float *>(smem + (e >> 1) * S::kRingBytes);
        if constexpr (S::kEarlyShared) return reinterpret_cast<float *>(smem + S::kEarlyOffset) + (e >> 1) * S::kSlotFloats;
        return slot_at(2 * chunks + cta * kWarps + (e >> 1));
    };

    // ---- this warp's share ----
    int stage = 0, step = 0;  // step: the lookup slot of this step's tile
    while (x < x_end) {       // one item's tiles
        const int row_tiles = prefix[here.row + 1] - prefix[here.row];
        const int n_tiles = min(row_tiles - here.tile, x_end - x);
        const bool whole = n_tiles == row_tiles;
        const int row = here.row, item = here.item;
        const bool more = x + n_tiles < x_end;

        if (!kQueriesAhead) load_queries(here);
        place_queries();
        float o[kSteps][NB][4];
        float m[NB][2], l[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            m[b][0] = m[b][1] = kNoMaximum;
            l[b][0] = l[b][1] = 0.0f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[s][b][i] = 0.0f;
        }

#pragma unroll 1
        for (int i = 0; i < n_tiles; ++i) {
            cp_async_wait<S::kStages - 1>();
            __syncwarp();
            const uint32_t st = ring + stage * S::kStageBytes;
            const uint32_t valid = sm_valid[warp][stage];
            // Chunk 2 s + e of a row whose swizzle is in `at` already.
            auto chunk_pair = [](uint32_t at, int s) {
                return kWide ? (at ^ ((s & 3) << 5)) + (s >> 2) * 128 : (at ^ ((s & 1) << 5)) + (s >> 1) * 64;
            };

            // Scores: rows = tokens lane / 4 and + 8 of each set, columns = heads
            // 2 (lane % 4) and + 1.
            constexpr int kChains = NB == 1 ? 2 : 1;  // shorter chains of dependent MMAs
            float sc[kSets][NB][4] = {}, sd[kSets][NB][4] = {};
            {
                const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
                const uint32_t at = st + r * S::kRowBytes + (((lane >> 4) ^ swizzle(r)) << 4);
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
                    for (int t = 0; t < kSets; ++t) {
                        uint32_t kf[4];
                        ldmatrix4(kf, chunk_pair(at, ks) + t * 16 * S::kRowBytes);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            mma16816(ks % kChains == 0 ? sc[t][b] : sd[t][b], kf, qf[ks][b][0], qf[ks][b][1]);
                    }
            }
            if (more && i == n_tiles - 1) {
                next_item(here);
                if (kQueriesAhead) load_queries(here);
            }
#pragma unroll
            for (int t = 0; t < kSets; ++t)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[t][b][e] = (kChains == 2 ? sc[t][b][e] + sd[t][b][e] : sc[t][b][e]) * a.scale_log2;
            if (valid != kAllSeen) {
#pragma unroll
                for (int t = 0; t < kSets; ++t)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!((valid >> (t * 16 + (e >> 1) * 8 + lane / 4)) & 1)) sc[t][b][e] = -INFINITY;
            }
            // The maximum m is kept until a score is 2^8 past it (weights up to 2^8 cost
            // nothing in FP32): most steps then need no maximum over the lanes, and no rescaling.
            float top[NB][2];
            bool past = false;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t = fmaxf(sc[0][b][e], sc[0][b][e + 2]);
                    if constexpr (kSets == 2) t = fmaxf(t, fmaxf(sc[kSets - 1][b][e], sc[kSets - 1][b][e + 2]));
                    top[b][e] = t;
                    past |= top[b][e] > m[b][e] + 8.0f;
                }
            if (__any_sync(0xFFFFFFFFu, past)) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = fmaxf(top[b][e], m[b][e]);
                        t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 4));
                        t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8));
                        t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
                        const float f = exp2_approx(m[b][e] - t);
                        m[b][e] = t;
                        l[b][e] *= f;
#pragma unroll
                        for (int s = 0; s < kSteps; ++s) {
                            o[s][b][e] *= f;
                            o[s][b][e + 2] *= f;
                        }
                    }
            }
            uint32_t hi[kSets][NB][2], lo[kSets][NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int t = 0; t < kSets; ++t) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = exp2_approx(sc[t][b][e] - m[b][e & 1]);
                        l[b][e & 1] += p[e];
                    }
                    // Tokens by heads -> heads by tokens, the B operand of the product with V.
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t h = __byte_perm(__float_as_uint(p[2 * e]), __float_as_uint(p[2 * e + 1]), 0x7632);
                        const uint32_t r = pack_bf16(rest_of(p[2 * e]), rest_of(p[2 * e + 1]));
                        hi[t][b][e] = movmatrix_trans(h);
                        lo[t][b][e] = movmatrix_trans(r);
                    }
                }
            }
            if (valid != 0) {  // a tile with nothing in it was not copied
                const int r = (lane & 7) + ((lane >> 4) & 1) * 8;
                const uint32_t at = st + (kSub + r) * S::kRowBytes + ((((lane >> 3) & 1) ^ swizzle(r)) << 4);
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int t = 0; t < kSets; ++t) {
                        uint32_t vf[4];
                        ldmatrix4_trans(vf, chunk_pair(at, s) + t * 16 * S::kRowBytes);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            mma16816(o[s][b], vf, hi[t][b][0], hi[t][b][1]);
                            mma16816(o[s][b], vf, lo[t][b][0], lo[t][b][1]);
                        }
                    }
            }
            __syncwarp();  // the stage is read: it takes the tile kStages on
            // That tile's lookup slot is one before this step's, mod kSlots; the one kStages
            // further is looked up now. (Keys refilled right after the scores, before the
            // softmax, came out slower: the copies' issue waits for the memory system.)
            fill(stage, step == 0 ? kSlots - 1 : step - 1);
            look_up(step < 2 ? step + kSlots - 2 : step - 2);
            cp_async_commit();  // a group a step, empty or not
            stage = stage + 1 == S::kStages ? 0 : stage + 1;
            step = step + 1 == kSlots ? 0 : step + 1;
        }

        // Sums over the lanes that share a column; the maxima are equal there already.
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[b][e] += __shfl_xor_sync(0xFFFFFFFFu, l[b][e], 4);
                l[b][e] += __shfl_xor_sync(0xFFFFFFFFu, l[b][e], 8);
                l[b][e] += __shfl_xor_sync(0xFFFFFFFFu, l[b][e], 16);
            }
        x += n_tiles;
        if (whole) {  // nobody else has tiles of this item
            const Heads heads = heads_of(row, item);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float inv0 = inverse(l[b][0]), inv1 = inverse(l[b][1]);
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    store_out(heads, s, b, o[s][b][0], o[s][b][1], o[s][b][2], o[s][b][3], inv0, inv1);
                if (lane < 4) {
                    store_lse(heads, b * 8 + lane * 2, m[b][0], l[b][0]);
                    store_lse(heads, b * 8 + lane * 2 + 1, m[b][1], l[b][1]);
                }
            }
        } else {
            const int entry = warp * 2 + (x == x_end ? 1 : 0);
            if (x == x_end) {  // into the ring: nothing but empty groups is on its way
                cp_async_wait<0>();
                __syncwarp();
            }
            float *to = entry_at(entry);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    reinterpret_cast<float4 *>(to)[(s * NB + b) * 32 + lane] =
                        make_float4(o[s][b][0], o[s][b][1], o[s][b][2], o[s][b][3]);
                if (lane < 4) {
                    float2 *ml = reinterpret_cast<float2 *>(to + S::kMaximaAt + b * 8) + lane;
                    ml[0] = make_float2(m[b][0], m[b][1]);
                    ml[S::kHeads / 2] = make_float2(l[b][0], l[b][1]);
                }
            }
            if (lane == 0) sm_key[entry] = row * items_per_row + item;
        }
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- join what the warps have left, item by item ----
    // Each warp takes its share of the fragments (16 values of 8 heads).
    constexpr int kPer = (kSteps + kWarps - 1) / kWarps, kJobs = kPer * NB;
    auto frag_of = [&](int job) { return (warp * kPer + job / NB) * NB + job % NB; };
    auto slot_of = [&](int first, int q) { return 2 * (first + q) + (q == 0 ? 1 : 0); };  // piece q of an item
    const int my_key = lane < 2 * kWarps ? sm_key[lane] : -1;
    unsigned alike = 0;  // entries of the same item
#pragma unroll
    for (int e = 0; e < 2 * kWarps; ++e)
        alike |= static_cast<unsigned>(__shfl_sync(0xFFFFFFFFu, my_key, e) == my_key) << e;
    unsigned items = __ballot_sync(0xFFFFFFFFu, my_key >= 0 && lane == __ffs(alike) - 1);
    // Items that other CTAs have pieces of too: at most the first and the last.
    struct Crossing {
        int key, first, pieces;
    };
    Crossing crossing[2] = {};
    int crossings = 0;
    for (; items != 0; items &= items - 1) {
        const int key = __shfl_sync(0xFFFFFFFFu, my_key, __ffs(items) - 1);
        const unsigned entries = __shfl_sync(0xFFFFFFFFu, alike, __ffs(items) - 1);
        const int row = quotient(key, items_per_row), item = key - row * items_per_row;
        const int row_tiles = prefix[row + 1] - prefix[row];
        const int item_x = prefix[row] * items_per_row + item * row_tiles;
        // Chunks first .. first + pieces - 1 hold a piece of this item each (a short one is in
        // one chunk, wherever the even cut would be).
        const bool within = row_tiles <= uncut;
        const int first = within ? cta : cut.owner(item_x);
        const int pieces = within ? 1 : cut.owner(item_x + row_tiles - 1) - first + 1;
        const Heads heads = heads_of(row, item);
        int dst = pieces == 1 ? -1 : slot_of(first, cta - first);
#pragma unroll 1
        for (int job = 0; job < kJobs; ++job) {
            const int frag = frag_of(job), h = frag % NB * 8 + (lane & 3) * 2;
            if (frag >= kSteps * NB) break;
            float2 mk[2 * kWarps], mm = make_float2(kNoMaximum, kNoMaximum), ll = make_float2(0.0f, 0.0f);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 2 * kWarps; ++e)
                if (entries >> e & 1) {
                    mk[e] = *reinterpret_cast<const float2 *>(entry_at(e) + S::kMaximaAt + h);
                    mm.x = fmaxf(mm.x, mk[e].x);
                    mm.y = fmaxf(mm.y, mk[e].y);
                }
#pragma unroll
            for (int e = 0; e < 2 * kWarps; ++e)
                if (entries >> e & 1) {
                    const float2 lk = *reinterpret_cast<const float2 *>(entry_at(e) + S::kMaximaAt + S::kHeads + h);
                    const float4 u = reinterpret_cast<const float4 *>(entry_at(e))[frag * 32 + lane];
                    const float f0 = exp2_approx(mk[e].x - mm.x), f1 = exp2_approx(mk[e].y - mm.y);
                    ll.x += f0 * lk.x;
                    ll.y += f1 * lk.y;
                    v.x += f0 * u.x; v.y += f1 * u.y; v.z += f0 * u.z; v.w += f1 * u.w;
                }
            const bool tell = frag < NB && lane < 4;  // the first fragment of a block of heads
            if (dst < 0) {
                store_out(heads, frag / NB, frag % NB, v.x, v.y, v.z, v.w, inverse(ll.x), inverse(ll.y));
                if (tell) {
                    store_lse(heads, h, mm.x, ll.x);
                    store_lse(heads, h + 1, mm.y, ll.y);
                }
            } else {
                float *to = slot_at(dst);
                __stcg(reinterpret_cast<float4 *>(to) + frag * 32 + lane, v);
                if (tell) {
                    __stcg(reinterpret_cast<float2 *>(to + S::kMaximaAt + h), mm);
                    __stcg(reinterpret_cast<float2 *>(to + S::kMaximaAt + S::kHeads + h), ll);
                }
            }
        }
        if (dst >= 0) crossing[crossings++ > 0 ? 1 : 0] = {key, first, pieces};
    }
    if (crossings == 0) return;

    // ---- join the chunks ----
    // Arrive, and the last of a group of chunks joins it; arrive, and the last group's
    // joiner joins the groups. Sources are added in order.
    auto arrive = [&](int first, int q, int level, int n) -> int {
        // Releases all threads' stores (a barrier orders them before it), acquires the other
        // CTAs'. The counter is zero again for the next call.
        unsigned *counter = a.counters + 2 * slot_of(first, q) + level;
        const bool last = ptx::atom_add_acq_rel_gpu(counter, 1u) + 1 == static_cast<unsigned>(n);
        if (last) *counter = 0u;
        return last;
    };
    auto group_size = [&](int pieces) {
        return pieces <= kAttnOneLevel ? kAttnOneLevel : static_cast<int>(ceilf(sqrtf(static_cast<float>(pieces))));
    };
    auto group_of = [&](int first, int size) { return quotient(cta - first, size) * size; };
    __syncthreads();  // every thread's stores are done
    if (tid % 32 == 0 && warp < crossings) {
        const Crossing &c = warp == 0 ? crossing[0] : crossing[1];
        const int size = group_size(c.pieces), q0 = group_of(c.first, size);
        sm_last[warp] = arrive(c.first, q0, 0, min(size, c.pieces - q0));
    }
    __syncthreads();
    for (int i = 0; i < crossings; ++i) {
        if (!sm_last[i]) continue;
        const int key = i == 0 ? crossing[0].key : crossing[1].key;
        const int first = i == 0 ? crossing[0].first : crossing[1].first;
        const int pieces = i == 0 ? crossing[0].pieces : crossing[1].pieces;
        const int row = quotient(key, items_per_row);
        const Heads heads = heads_of(row, key - row * items_per_row);
        float *factor = reinterpret_cast<float *>(smem + S::kFactorOffset);
        float *sm_m = reinterpret_cast<float *>(smem + S::kMlOffset), *sm_l = sm_m + S::kHeads;
        const int size = group_size(pieces), groups = quotient(pieces + size - 1, size);
        int q0 = group_of(first, size), q_step = 1, n = min(size, pieces - q0);
        for (int level = 0; level < 2; ++level) {
            if (level == 1) {
                __syncthreads();  // every thread's stores are done
                if (tid == 0) sm_last[2] = arrive(first, 0, 1, groups);
                __syncthreads();
                if (!sm_last[2]) break;
                q0 = 0;
                q_step = size;
                n = groups;
            }
            const int dst = level == 1 || groups == 1 ? -1 : slot_of(first, q0);
            auto source = [&](int k) { return slot_at(slot_of(first, q0 + k * q_step)); };

            // A lane is a source for the factors; the first fragments are on their way
            // meanwhile.
            constexpr int kPair = kJobs > 1 ? 2 : 1, kBatch = 12;
            float4 u[kPair][kBatch];
            auto load = [&](int job, int k0) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
#pragma unroll
                    for (int j = 0; j < kPair; ++j)
                        if (k0 + k < n && job + j < kJobs && frag_of(job + j) < kSteps * NB)
                            u[j][k] = __ldcg(reinterpret_cast<const float4 *>(source(k0 + k)) + frag_of(job + j) * 32 + lane);
            };
            {
                constexpr int kMine = S::kHeads / kWarps;  // heads of a warp
                float mk[kMine], lk[kMine], mm[kMine];
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const float *src = source(min(lane, n - 1)) + S::kMaximaAt + warp * kMine + i;
                    mm[i] = mk[i] = lane < n ? __ldcg(src) : kNoMaximum;
                    lk[i] = lane < n ? __ldcg(src + S::kHeads) : 0.0f;
                }
                load(0, 0);
#pragma unroll
                for (int s = 16; s > 0; s >>= 1)
#pragma unroll
                    for (int i = 0; i < kMine; ++i) mm[i] = fmaxf(mm[i], __shfl_xor_sync(0xFFFFFFFFu, mm[i], s));
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const float f = exp2_approx(mk[i] - mm[i]);
                    if (lane < n) factor[lane * S::kHeads + warp * kMine + i] = f;
                    lk[i] *= f;
                }
#pragma unroll
                for (int s = 16; s > 0; s >>= 1)
#pragma unroll
                    for (int i = 0; i < kMine; ++i) lk[i] += __shfl_xor_sync(0xFFFFFFFFu, lk[i], s);
                if (lane == 0)
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        sm_m[warp * kMine + i] = mm[i];
                        sm_l[warp * kMine + i] = lk[i];
                    }
            }
            __syncthreads();
#pragma unroll 1
            for (int job = 0; job < kJobs; job += kPair) {
                float v[kPair][4] = {};
#pragma unroll 1
                for (int k0 = 0; k0 < n; k0 += kBatch) {
                    if (job + k0 > 0) load(job, k0);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        if (k0 + k >= n) break;
#pragma unroll
                        for (int j = 0; j < kPair; ++j) {
                            const int h = frag_of(job + j) % NB * 8 + (lane & 3) * 2;
                            const float2 f = *reinterpret_cast<const float2 *>(factor + (k0 + k) * S::kHeads + h);
                            v[j][0] += f.x * u[j][k].x;
                            v[j][1] += f.y * u[j][k].y;
                            v[j][2] += f.x * u[j][k].z;
                            v[j][3] += f.y * u[j][k].w;
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < kPair; ++j) {
                    const int frag = frag_of(job + j), h = frag % NB * 8 + (lane & 3) * 2;
                    if (job + j >= kJobs || frag >= kSteps * NB) continue;
                    if (dst >= 0)
                        __stcg(reinterpret_cast<float4 *>(slot_at(dst)) + frag * 32 + lane,
                               make_float4(v[j][0], v[j][1], v[j][2], v[j][3]));
                    else
                        store_out(heads, frag / NB, frag % NB, v[j][0], v[j][1], v[j][2], v[j][3], inverse(sm_l[h]),
                                  inverse(sm_l[h + 1]));
                }
            }
            if (tid < S::kHeads) {
                if (dst >= 0) {
                    __stcg(slot_at(dst) + S::kMaximaAt + tid, sm_m[tid]);
                    __stcg(slot_at(dst) + S::kMaximaAt + S::kHeads + tid, sm_l[tid]);
                } else {
                    store_lse(heads, tid, sm_m[tid], sm_l[tid]);
                }
            }
            if (dst < 0) break;
        }
        __syncthreads();  // the factors are used again
    }
}

template <int D, int NB, int FORM>
cudaError_t launch(const ArgsOf<FORM> &a, int num_sms, int device, cudaStream_t stream, bool pdl) {
    using S = Shape<D, NB>;
    static bool configured[64] = {};
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    if (!configured[device]) {
        cudaError_t e = cudaFuncSetAttribute(decode_attention_kernel<D, NB, FORM>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes(kAttnMaxRows));
        if (e != cudaSuccess) return e;
        configured[device] = true;
    }
    // No more CTAs than the tables could ever hold tiles for their warps.
    long long tokens = a.capacity;
    if constexpr (FORM == kJoined) tokens += a.prefix_capacity;
    const long long tiles = static_cast<long long>(a.rows) * a.kv_heads * a.head_blocks * ((tokens + S::kSub - 1) / S::kSub);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(num_sms * attn_ctas_per_sm(D, NB), (tiles + kWarps - 1) / kWarps)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = S::bytes(a.rows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, decode_attention_kernel<D, NB, FORM>, a);
}

template <int D, int FORM>
cudaError_t launch_dim(const ArgsOf<FORM> &a, int num_sms, int device, cudaStream_t stream, bool pdl) {
    if (a.block_heads <= 8) return launch<D, 1, FORM>(a, num_sms, device, stream, pdl);
    if (a.block_heads <= 16) return launch<D, 2, FORM>(a, num_sms, device, stream, pdl);
    if constexpr (D <= 128) return launch<D, 4, FORM>(a, num_sms, device, stream, pdl);
    return cudaErrorInvalidValue;
}

template <int FORM>
cudaError_t launch_any_dim(const ArgsOf<FORM> &a, int head_dim, int num_sms, int device, cudaStream_t stream,
                           bool pdl) {
    switch (head_dim) {
        case 64: return launch_dim<64, FORM>(a, num_sms, device, stream, pdl);
        case 96: return launch_dim<96, FORM>(a, num_sms, device, stream, pdl);
        case 128: return launch_dim<128, FORM>(a, num_sms, device, stream, pdl);
        case 192: return launch_dim<192, FORM>(a, num_sms, device, stream, pdl);
        case 256: return launch_dim<256, FORM>(a, num_sms, device, stream, pdl);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t error_word(int **word) { return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_attn_err); }

}  // namespace
}  // namespace skinny
