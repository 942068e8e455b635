// Work split of the attention over a shared prefix (shared by the host and the kernels).
//
// The query rows of a key head are all rows' heads that share it, row-major: query row
// i = row * group + head. A unit is one key head with up to 128 (or 2 x 128) of its query
// rows; a step is one tile of the prefix's tokens for one unit. The steps of all units in
// (key head, block of query rows, tile) order are one sequence, cut evenly into one range per
// CTA. A CTA leaves a partial result for every unit that its range touches: the c-th CTA's
// part of unit u goes to slot c + u, which no other pair has (from one pair to the next in
// order, either c or u grows by one). The prefix's length lives on the device, so
// the kernels work the split out for themselves.
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
// tokens for two tiles of wide heads. 64 from 192 on, whose keys and values fill the ring
// otherwise.
__host__ __device__ constexpr int prefix_tokens(int head_dim, int tiles) {
    return head_dim > 128 ? 64 : tiles == 1 || head_dim <= 64 ? 128 : head_dim <= 96 ? 96 : 80;
}

struct PrefixPlan {
    int tokens;  // of a step
    int blocks;  // blocks of query rows of a key head
    int units;   // key heads * blocks
};
__host__ __device__ inline PrefixPlan prefix_plan(int rows, int group, int kv_heads, int head_dim) {
    const long long q = static_cast<long long>(rows) * group;
    const int tiles = prefix_tiles(head_dim, q), per = kPrefixRows * tiles;
    PrefixPlan p;
    p.tokens = prefix_tokens(head_dim, tiles);
    p.blocks = static_cast<int>((q + per - 1) / per);
    p.units = p.blocks * kv_heads;
    return p;
}

// CTAs that take part, of `grid`, for `total` steps.
__host__ __device__ inline int prefix_ctas(int grid, int total) { return total < grid ? total : grid; }
// First step of CTA c's range, and the CTA that a step is in.
__host__ __device__ inline int prefix_begin(int total, int ctas, int c) {
    return static_cast<int>(static_cast<long long>(total) * c / ctas);
}
__host__ __device__ inline int prefix_owner(int total, int ctas, int x) {
    return static_cast<int>(((static_cast<long long>(x) + 1) * ctas - 1) / total);
}

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
    const PrefixPlan p = prefix_plan(rows, q_heads / kv_heads, kv_heads, head_dim);
    const size_t heads = static_cast<size_t>(rows) * q_heads;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    PrefixWorkspace w;
    w.own_out = up(attn_workspace_bytes(sms));
    w.own_lse = w.own_out + up(heads * head_dim * sizeof(float));
    w.slots = w.own_lse + up(heads * sizeof(float));
    w.bytes = w.slots + (static_cast<size_t>(sms) + p.units) * prefix_slot_floats(head_dim, q) * sizeof(float);
    return w;
}

}  // namespace skinny
