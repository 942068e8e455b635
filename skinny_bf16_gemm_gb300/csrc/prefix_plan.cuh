// Work split of the attention over a shared prefix (shared by the host and the kernels).
//
// The query rows of a key head are all rows' heads that share it, row-major: query row
// i = row * group + head; 128 or 2 x 128 of them are a block. A step is one tile of the
// prefix's tokens for one block. The tiles of all key heads, in (key head, tile) order, are
// one sequence, cut evenly into ranges; a range is gone through by one CTA for each block (or
// for each of `lanes` blocks at a time, if there are more blocks than CTAs), all at the same
// time, so that the keys and values that they share come from HBM once. A CTA leaves a partial
// result for every key head that its range touches: range r's part of key head h goes to slot
// (r + h) * blocks + block, and no two pairs have the same r + h (from one pair to the next in
// order, either r or h grows by one). The prefix's length lives on the device, so the
// kernels work the cut out for themselves.
#pragma once

#include <cstddef>
#include <cstdint>

#include "attention_plan.cuh"

namespace skinny {

constexpr int kPrefixRows = 128;  // query rows of a tile: the MMA's M

// Tiles of 128 query rows a CTA has at once: two, whose softmaxes and products take turns,
// where there are that many rows and the tensor memory holds both.
__host__ __device__ constexpr int prefix_tiles(int head_dim, long long query_rows) {
    return head_dim <= 128 && query_rows > kPrefixRows ? 2 : 1;
}

// Tokens of a step. In tensor memory (512 columns) every tile has a place for its scores (one
// column a token), one for its weights (half a column) and one for its output (head_dim
// columns), all apart, so that the next scores are computed while the softmax runs: 80 or 96
// tokens for two tiles (96 are as many as a softmax thread has registers for). 64 from 192 on,
// whose keys and values fill the ring otherwise.
__host__ __device__ constexpr int prefix_tokens(int head_dim, int tiles) {
    return head_dim > 128 ? 64 : tiles == 1 ? 128 : head_dim <= 96 ? 96 : 80;
}

struct PrefixPlan {
    int tokens;  // of a step
    int blocks;  // blocks of query rows of a key head
};
__host__ __device__ inline PrefixPlan prefix_plan(int rows, int group, int head_dim) {
    const long long q = static_cast<long long>(rows) * group;
    const int tiles = prefix_tiles(head_dim, q), per = kPrefixRows * tiles;
    PrefixPlan p;
    p.tokens = prefix_tokens(head_dim, tiles);
    p.blocks = static_cast<int>((q + per - 1) / per);
    return p;
}

// Blocks that are gone through side by side with `ctas` CTAs, and the most ranges.
__host__ __device__ inline int prefix_lanes(int blocks, int ctas) {
    const int passes = (blocks + ctas - 1) / ctas;
    return (blocks + passes - 1) / passes;
}
__host__ __device__ inline int prefix_ranges(int blocks, int ctas) { return ctas / prefix_lanes(blocks, ctas); }

// CTAs for the prefix where the rows' own tokens have the other SMs at the same time, or `sms`:
// one after the other on all of them. Side by side hides the shorter kernel's start and end, some
// 7 us, but the SMs are dealt out by what the tables could hold, the lengths being on the device:
// the steps of the prefix (0.9 us for one on the tensor cores, 1.2 with wide heads) and half the
// rows' own tokens (at 6.8 TB/s), each with 1.5 us more for what does not shrink with more SMs. Up
// to 20 us in all even lengths of 0 or of the whole table cost no more than is hidden; beyond, they
// might. 64 rows x 7 heads behind 16001 tokens, 1000 of their own: 23.7 us side by side, 30.4 one
// after the other; 60001 and 1000: 30.6, 38.7; 16001 and 4000: 31.4, 41.6; 32 rows x 32 heads of 64
// over 8, 32768 and 300: 33.7, 42.8; 16 rows x 7, 16001 and 300: 17.7 either way; 64 x 56 over 8,
// 65521 and 1000, 100 us in all: 163.7 side by side at the best, 158.9 one after the other.
inline int prefix_ctas(int rows, int kv_heads, int head_dim, const PrefixPlan &plan, long long prefix_tokens,
                       long long own_tokens, int sms) {
    const double steps = static_cast<double>((prefix_tokens + plan.tokens - 1) / plan.tokens) * kv_heads * plan.blocks;
    const double prefix = steps * (head_dim > 128 ? 1.2 : 0.9) / sms;
    const double own = static_cast<double>(own_tokens) * rows * kv_heads * head_dim * 2 / 6.8e6;
    if (prefix + own > 20.0) return sms;
    const int ctas = static_cast<int>(sms * (prefix + 1.5) / (prefix + own + 3.0));
    return ctas < 1 ? 1 : ctas;
}

// An even cut of `total` tiles into ranges, `most` at most: the first `extra` have base + 1.
struct PrefixCut {
    int ranges, base, extra;
    __host__ __device__ PrefixCut(int total, int most) {
        ranges = total < most ? total : most;
        base = ranges > 0 ? total / ranges : 0;
        extra = total - base * ranges;
    }
    __host__ __device__ int begin(int r) const { return r * base + (r < extra ? r : extra); }
    __host__ __device__ int owner(int x) const {
        const int at = extra * (base + 1);
        return x < at ? x / (base + 1) : extra + (x - at) / base;
    }
};

// How a tile's tokens lie in shared memory: rows of 128 bytes (64 values, a chunk) in swizzle
// atoms of 8 tokens. Where heads are whole chunks the chunks of 8 tokens lie side by side, so that
// one copy brings them all; else (96) all tokens' first chunks come before their second ones.
constexpr bool prefix_merged(int head_dim) { return head_dim % 64 == 0; }

// The ring of a CTA's tiles of keys and values. They come in turn, keys first: unit 2 t is tile t's
// keys, 2 t + 1 its values. Keys and values have stages of their own: a loader waits for the
// phase in which a stage comes free by its parity, so it must know that the phase before is
// complete, and it does where it waited for that itself before its last unit there. An even number
// of stages, gone through in the order of the units, is such a ring. An odd one is not: there the
// unit before is the other kind's, and of the one before that nothing is known but that it came
// earlier (the scores of a later tile may be complete sooner than the product with its values), so
// the odd stage is the keys', which are wanted first.
template <int kStages>
struct PrefixRing {
    static constexpr int kKeys = (kStages + 1) / 2, kValues = kStages / 2;
    // The stage of a unit, and how many units of the ring it had before.
    __host__ __device__ static constexpr int stage(int unit) {
        if (kStages % 2 == 0) return unit % kStages;
        return unit % 2 ? kKeys + unit / 2 % kValues : unit / 2 % kKeys;
    }
    __host__ __device__ static constexpr int round(int unit) {
        return kStages % 2 == 0 ? unit / kStages : unit / 2 / (unit % 2 ? kValues : kKeys);
    }
    // The first of a kind's units whose copies may be on their way when `end` is the kind's next
    // one: before a later one was put into its stage each one before was waited for.
    __host__ __device__ static constexpr int first_on_its_way(int end) {
        const int kind = end % 2, first = end - 2 * (kind ? kValues : kKeys);
        return first > kind ? first : kind;
    }
};

// A partial: for each query row of the unit head_dim sums, then all maxima, then all sums of
// weights.
__host__ __device__ inline size_t prefix_slot_floats(int head_dim, long long query_rows) {
    return static_cast<size_t>(kPrefixRows) * prefix_tiles(head_dim, query_rows) * (head_dim + 2);
}

// The workspace: that of the rows' own tokens (attention_plan.cuh), those tokens' results in
// FP32 and their log-sums, then the slots.
struct PrefixWorkspace {
    size_t own_out, own_lse, slots, bytes;  // byte offsets, and the end
};
inline PrefixWorkspace prefix_workspace(int rows, int q_heads, int kv_heads, int head_dim, int sms) {
    const long long q = static_cast<long long>(rows) * (q_heads / kv_heads);
    const PrefixPlan p = prefix_plan(rows, q_heads / kv_heads, head_dim);
    // The slots grow with the blocks, so that a workspace does for fewer rows too: at most
    // sms + key heads * blocks.
    const size_t slots = static_cast<size_t>(sms) + static_cast<size_t>(kv_heads) * p.blocks;
    const size_t heads = static_cast<size_t>(rows) * q_heads;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    PrefixWorkspace w;
    w.own_out = up(attn_workspace_bytes(sms));
    w.own_lse = w.own_out + up(heads * head_dim * sizeof(float));
    w.slots = w.own_lse + up(heads * sizeof(float));
    w.bytes = w.slots + slots * prefix_slot_floats(head_dim, q) * sizeof(float);
    return w;
}

}  // namespace skinny
