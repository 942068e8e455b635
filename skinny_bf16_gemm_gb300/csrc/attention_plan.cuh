// Work split of the decode attention (shared by the host and the kernel).
//
// An item is one row's key head with up to 32 of the query heads that share it (a
// head block). What an item sees of its row's cache is cut into tiles of one warp step
// (16 or 32 tokens). The tiles of all items in (row, key head, head block, tile) order
// are one sequence, cut evenly into one chunk per CTA and each chunk evenly into the
// shares of its warps, so that every warp streams the same number of bytes whatever the
// lengths are. The lengths live on the device, so each CTA works the split out for itself.
#pragma once

#include <cstddef>
#include <cstdint>

namespace skinny {

constexpr int kAttnMinTile = 16;    // tokens of the smallest tile
constexpr int kAttnMaxRows = 1024;  // rows whose prefix sums a CTA keeps
constexpr int kAttnWarps = 4;
// Partials of an item that are joined at once; more are joined in groups (16 rows to 2000,
// 16 heads of 128: 19.0 us, 22.2 in groups from 13 on; two items of 32 parts, 256-wide:
// 23.8 us in groups, 37.8 at once).
constexpr int kAttnOneLevel = 20;
constexpr int kAttnMaxSms = 256;    // SMs used: groups of up to 23 of 512 CTAs

inline int attn_sms(int num_sms) { return num_sms < kAttnMaxSms ? num_sms : kAttnMaxSms; }

// Query heads of a head block: 8 * NB columns of the MMA, NB as far as the
// accumulators (NB * D / 4 registers a thread) go.
__host__ __device__ inline int attn_max_nb(int head_dim) { return head_dim <= 128 ? 4 : 2; }

// Two CTAs an SM where the rings fit and a warp's step leaves gaps: small heads (64 ragged
// rows to 16384 of 64-wide heads, pages by head: 163 us, 194 with one CTA and more stages),
// and many query heads to a key head (16 rows to 8192, 128-wide, 16 heads: 43 us, 50 with
// one; 32 heads: 67, 83 with one). One for 192-wide heads, 16 to a key head: 45 us, 49 with
// two, whose copies queue too long.
constexpr int attn_ctas_per_sm(int head_dim, int nb) { return head_dim <= 64 || (nb > 1 && head_dim <= 128) ? 2 : 1; }

// A partial: heads * head_dim sums, then the heads' maxima and sums of weights. Every
// CTA has two slots for its chunk's (of an item that began before it, and of one that
// goes on after it or only it has a part of) and one for each warp.
constexpr int attn_slot_floats(int head_dim, int nb) { return 8 * nb * (head_dim + 2); }
constexpr int attn_slots_per_cta() { return 2 + kAttnWarps; }

// The workspace: two counters for each of the chunks' slots (all zero between calls), in
// a space that does for the largest grid, then the slots.
constexpr size_t kAttnCounterBytes = static_cast<size_t>(2 * 2 * 2) * kAttnMaxSms * sizeof(unsigned);
inline size_t attn_workspace_bytes(int sms) {
    constexpr int dims[] = {64, 96, 128, 192, 256};
    size_t most = 0;
    for (int d : dims)
        for (int nb = 1; nb <= attn_max_nb(d); nb *= 2) {
            const size_t n = static_cast<size_t>(attn_ctas_per_sm(d, nb)) * attn_slots_per_cta() * attn_slot_floats(d, nb);
            if (n > most) most = n;
        }
    return kAttnCounterBytes + most * sms * sizeof(float);
}

}  // namespace skinny
