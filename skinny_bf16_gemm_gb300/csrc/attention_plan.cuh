// Work split of the decode attention (shared by the host and the kernel).
//
// An item is one row's key head with up to 32 of the query heads that share it (a
// head block). What an item sees of its row's cache is cut into tiles of 64
// tokens, the tiles of all items in (row, key head, head block, tile) order are one
// sequence, and the sequence is cut into contiguous ranges of (almost) equal length,
// one per CTA: every CTA streams the same number of bytes whatever the lengths are.
// The lengths live on the device, so each CTA works the split out for itself.
#pragma once

#include <cstdint>

namespace skinny {

constexpr int kAttnTile = 64;          // tokens per tile: 16 for each of the 4 warps
constexpr int kAttnMaxRows = 1024;     // rows whose prefix sums a CTA keeps
constexpr int kAttnGroup = 16;         // partials one CTA joins at a time
constexpr int kAttnCtasPerSm = 2;
constexpr int kAttnMaxHeads = 32;      // query heads of one head block
constexpr int kAttnSlotFloats = 4096 + 2 * kAttnMaxHeads;  // heads * head_dim, then m and l

// Query heads of a head block: 8 * NB columns of the MMA, NB as far as the
// accumulators (NB * D / 4 registers a thread) go.
__host__ __device__ inline int attn_max_nb(int head_dim) { return head_dim <= 128 ? 4 : 2; }

constexpr int kAttnMaxSms = 192;       // SMs used: two levels of joins reach 24 * 16 CTAs
inline int attn_sms(int num_sms) { return num_sms < kAttnMaxSms ? num_sms : kAttnMaxSms; }

// Largest grid and the workspace that goes with it: the counters first (two per
// slot, zero between calls), then the partial slots (two per CTA).
inline int attn_max_ctas(int num_sms) { return num_sms * kAttnCtasPerSm; }
inline size_t attn_counter_bytes(int ctas) {
    return (static_cast<size_t>(4) * ctas * sizeof(unsigned) + 255) / 256 * 256;
}
inline size_t attn_workspace_bytes(int num_sms) {
    const int ctas = attn_max_ctas(num_sms);
    return attn_counter_bytes(ctas) + static_cast<size_t>(2) * ctas * kAttnSlotFloats * sizeof(float);
}

}  // namespace skinny
