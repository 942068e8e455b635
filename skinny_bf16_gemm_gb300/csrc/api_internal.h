// What the files of the C ABI share: the per-device state, the launch settings of a call
// and the argument checks (api.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernels.h"
#include "skinny.h"

namespace skinny {

constexpr int kMaxDevices = 64;
constexpr int kMaxHeads = 1024;

struct DeviceState {
    bool ready = false;
    int sms = 0;
    int major = 0, minor = 0;
    // Split-K scratch of the decode GEMM, sized for one CTA per SM.
    void *scratch = nullptr;
    float *partials = nullptr;
    unsigned *flags = nullptr;
    int *err = nullptr;
    size_t flag_bytes = 0;
    // decode_gemm_bf16_reduce_rmsnorm's "its GEMM is complete" word (in the
    // scratch's last 256 bytes, after the error word).
    unsigned *gemm_done = nullptr;
    float *lora_sums = nullptr;  // decode_gemm_bf16_lora's A x, kLoraScratchFloats
    // A host-mapped word the decode GEMM sets when one of its waits runs out:
    // the host reads it without synchronising, so the next call can refuse to
    // run on scratch a kernel left half used (host_err) -- and the kernel's
    // address of it (host_err_dev).
    int *host_err = nullptr;
    int *host_err_dev = nullptr;
};

// The current device's index, and its state (SKINNY_ERR_DEVICE if it is no sm_103).
int current_device(int *dev);
int device_state(int dev, DeviceState **out);
// The pointer must be device (or managed) memory of device `dev`.
int check_device_pointer(const void *p, int dev);

// The launch settings of one call: the caller's options where given, else the
// process-wide settings (skinny_set_pdl, skinny_set_l2_prefetch).
struct LaunchSettings {
    bool pdl;
    int l2_lead;
    int l2_after_reduce;
};
int resolve_settings(const skinny_launch_opts *opts, LaunchSettings *out);

// A tensor map over a cache's keys or values with 128-byte swizzle; false if there is none for
// its strides. merged: [pages, groups of 8 tokens, chunks of 64 values (of all heads), 8, 64],
// boxes of box_rows tokens with the chunks of one head side by side in every group. Else
// [pages, heads, tokens, head_dim], boxes of box_rows tokens by 64 values.
bool encode_cache_map(CUtensorMap *map, const void *base, const skinny_kv_cache *c, int box_rows, bool merged);

// A cache's own rules, and the bytes its keys (or values) span.
int check_cache(const skinny_kv_cache *c, bool write, size_t *span);

// decode_attention_bf16's rules that need no device, and its kernel's arguments.
int check_attention(const skinny_decode_attention_args *p, size_t *pool);
void attention_args(const skinny_decode_attention_args *p, size_t pool, AttentionArgs *out);

inline bool overlaps(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bn && b0 < a0 + an;
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int log2_or_minus_one(int n) { return (n & (n - 1)) == 0 ? __builtin_ctz(n) : -1; }

// Bytes from a row's first element to past the last row's last.
inline size_t row_span(int rows, long long stride, long long width) {
    return (static_cast<size_t>(rows - 1) * stride + width) * 2;
}

}  // namespace skinny
