// Launch interface between the C ABI (api.cu) and the kernel translation units.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "epilogue.cuh"

namespace skinny {

// Bits of the device error word (one per waiting role that gave up).
enum ErrorBits : int {
    kErrProducerWait = 1,   // TMA producer: a pipeline slot never came free
    kErrMmaFullWait = 2,    // MMA issuer: a stage's copies never landed
    kErrMmaAccWait = 4,     // MMA issuer: the epilogue never released an accumulator
    kErrEpilogueWait = 8,   // epilogue: an accumulator never completed
    kErrDrain = 16,         // teardown: in-flight copies or MMAs did not finish
    kErrSelftest = 32,      // the watchdog self-test's deliberate wait ran out
    kErrUnknown = 64,       // the host-mapped word was set but the device word was not
    kErrReduceExchange = 128,  // reduce: a cluster exchange wait ran out
    kErrIndex = 256,  // a position, slot, length or page index on the device was out of range
    kErrPrefixWait = 512,  // attention over a shared prefix: a wait ran out
};

// Low-rank adapters beside a decode GEMM (decode_gemm_bf16_lora): row m's adapter is
// adapters[m], none if it is negative.
constexpr int kLoraMaxRank = 128;
constexpr int kLoraScratchFloats = 1 << 16;
struct LoraArgs {
    const uint16_t *A;    // [count][rank][K]
    const uint16_t *B;    // [count][N][rank]
    const int *adapters;  // [M]
    const float *scales;  // [count] or nullptr: 1
    int count, rank;
    int splits;   // K slices of A x
    float *sums;  // [splits][M][rank] FP32, rows without an adapter unwritten
};

struct GemmArgs {
    int M, N, K;
    uint16_t *out;          // [M, N] BF16 patterns
    float *partials;        // [2 * ctas][slot rows][128] FP32 split-K partial tiles
    int slot_floats;        // floats from one partial tile to the next
    unsigned *flags;        // [2 * ctas] "partial published" flags, zero between calls
    int *err;               // device error word
    int *host_err;          // host-mapped word set to 1 on any error, or nullptr
    unsigned long long wait_limit_ns;
    int selftest;           // 1: the MMA role waits on a barrier nothing completes
    // lm_head epilogue (logits = 1): v = soft_cap > 0 ? soft_cap * tanh(v / soft_cap)
    // : v; v *= scale; applied to the FP32 sum before the one BF16 rounding.
    int logits;
    float soft_cap, scale;
    // 1: every piece, whole tiles included, leaves its FP32 partial in its scratch
    // slot and nothing is finished here (no flags): the reduce kernel that follows
    // adds them (decode_gemm_bf16_reduce_rmsnorm).
    int publish_only;
    // Deep ring only: weight blocks each CTA prefetches into L2, beyond its ring's
    // first fill, before waiting on the previous kernel (skinny_set_l2_prefetch).
    int l2_lead;
    // The "GEMM before the reduce is complete" word of decode_gemm_bf16_reduce_rmsnorm
    // (set by its reduce, cleared by its GEMM), or nullptr. With l2_after_reduce > 0
    // the producer waits (bounded) for it to be set and then prefetches that many
    // more weight blocks into L2 before waiting on the previous kernel.
    unsigned *gemm_done;
    int l2_after_reduce;
    int clear_gemm_done;  // 1: clear the word once the previous kernel is complete
    // epilogue = 1: bias, activation and residual (epilogue.cuh) on the FP32 sum.
    int epilogue;
    Epilogue epi;
    // lora.rank > 0: the adapters' second half, added to the FP32 sum before the epilogue.
    LoraArgs lora;
};

// Default and largest l2_lead. Measured on GB300: 6 suits back-to-back GEMMs
// (each CTA's early blocks arrive while the previous kernel's last CTAs finish);
// 0 suits a GEMM behind a short latency-bound kernel, such as the layer chain's
// reduce, where those requests only slow the previous GEMM's last CTAs.
constexpr int kL2LeadDefault = 6;
constexpr int kL2LeadMax = 64;

// Where the reduce kernel finds a publish-only GEMM's partials of the 7168
// slot-0 columns: the GEMM's geometry (tiles, K blocks, CTAs) and scratch.
struct SplitKPartials {
    const float *partials;  // [2 * ctas][slot_floats]
    int slot_floats;
    int M, N, K, ctas;
    unsigned *gemm_done;    // set to 1 once the GEMM is complete (or nullptr)
};

// Pipeline depth and shared memory of the decode GEMM for a padded row count,
// with the shallow or the deep ring (plan.cuh use_shallow_ring).
int gemm_stages(int mma_n, bool shallow);
int gemm_smem_bytes(int mma_n, bool shallow);

// Launch the decode GEMM: grid = ctas CTAs of 192 threads; pdl sets the
// programmatic-dependent-launch attribute, shallow picks the ring.
cudaError_t launch_decode_gemm(const CUtensorMap &w_map, const CUtensorMap &x_map,
                               const GemmArgs &args, int mma_n, int ctas, cudaStream_t stream,
                               bool pdl, bool shallow, int device);

// The adapters' first half (lora_shrink.cu): K slices for a call, and l.sums from x.
int lora_splits(int M, int K, int rank, int num_sms);
cudaError_t launch_lora_shrink(const void *x, const LoraArgs &l, int M, int K, int num_sms, cudaStream_t stream,
                               bool pdl);
cudaError_t lora_error_word(int **word);

// Split-K scratch held in a static device array (decode_gemm_bf16_noalloc).
constexpr int kStaticScratchCtas = 160;   // CTAs the array holds partial tiles for
constexpr int kStaticSlotRows = 32;       // rows of x a static partial tile holds

struct StaticScratch {
    float *partials;      // [2 * max_ctas][kStaticSlotRows][128] FP32
    unsigned *flags;      // [2 * max_ctas], contiguous with err
    int *err;             // error word, right after the flag space
    size_t zero_bytes;    // bytes from `flags` through `err` that must start at zero
    int max_ctas;
};

// Device addresses of the static scratch on the current device; the first call
// per device looks them up (cudaGetSymbolAddress).
cudaError_t static_scratch_for_current_device(StaticScratch *out);

// Launch reduce + residual + RMSNorm over rows of 7168: M clusters of
// ctas_per_row CTAs.
cudaError_t launch_reduce_rmsnorm(const void *partials, int TP, const void *residual,
                                  const void *gamma, void *out, void *residual_out, int M,
                                  float eps, int ctas_per_row, cudaStream_t stream, bool pdl);

// Finish a publish-only decode GEMM: out[M, N] = the partials added in K order,
// rounded once to BF16, after the epilogue's steps if epi is given.
cudaError_t launch_splitk_finish(const SplitKPartials &fix, uint16_t *out, const Epilogue *epi,
                                 cudaStream_t stream, bool pdl);

// The same with slot 0 made from a publish-only GEMM's FP32 partials (added in
// K order, rounded once, and written to slot 0 of `partials`).
cudaError_t launch_reduce_rmsnorm_splitk(void *partials, int TP, const void *residual,
                                         const void *gamma, void *out, void *residual_out, int M,
                                         float eps, int ctas_per_row, const SplitKPartials &fix,
                                         cudaStream_t stream, bool pdl);

// The plain reduce with 8-CTA clusters whose last CTA keeps its sum of squares
// to itself, every exchange wait limited to limit_ns: the failure-path
// self-test (the waits run out, are recorded in the reduce's error word and
// end; the outputs are unspecified).
cudaError_t launch_reduce_rmsnorm_selftest(const void *partials, int TP, const void *residual,
                                           const void *gamma, void *out, void *residual_out,
                                           int M, float eps, unsigned long long limit_ns,
                                           cudaStream_t stream);

// Where the reduce keeps its own error word on the current device (nonzero: a cluster
// exchange wait ran out); the further kernels' below likewise.
cudaError_t reduce_error_word(int **word);

// Gather TP shards [TP, M, S] into rows [M, TP * S] (S a multiple of 8).
cudaError_t launch_gather(const void *shards, int TP, int M, int S, void *out,
                          cudaStream_t stream, bool pdl);

// Per-head norm, rotation and cache append (qk_norm_rope_bf16). Strides in elements.
struct RopeArgs {
    const uint16_t *qkv;  // rows of q heads, key heads, value heads
    long long qkv_stride;
    int rows, q_heads, kv_heads, head_dim;
    const uint16_t *q_gamma, *k_gamma;  // [head_dim] or nullptr: no norm
    float eps, inv_dim;  // inv_dim: 1 / head_dim
    const float *rope;  // [max_pos][rot_dim]: rot_dim / 2 cosines, then sines
    int max_pos, rot_dim, interleaved;
    const int *positions;
    uint16_t *q_out;
    long long q_stride;
    uint16_t *k_out;  // or nullptr
    long long k_stride;
    uint16_t *k_cache, *v_cache;  // both or neither
    int page_size, page_shift;  // page_shift: log2(page_size), or -1
    long long num_slots;        // pages * page_size
    long long page_stride, token_stride, head_stride;
    const long long *slots;
};
cudaError_t launch_qk_norm_rope(const RopeArgs &a, int num_sms, cudaStream_t stream, bool pdl);
cudaError_t rope_error_word(int **word);

// Decode attention over a paged cache (decode_attention_bf16). Strides in elements.
struct AttentionArgs {
    const uint16_t *q;  // rows of q_heads * head_dim
    long long q_stride;
    const uint16_t *k, *v;
    int num_pages, page_size;
    int page_shift;  // log2(page_size), or -1
    long long page_stride, token_stride, head_stride;
    const int *block_table;  // [rows][capacity / page_size]
    long long table_stride;
    const int *lengths;
    int rows, q_heads, kv_heads;
    int group;        // query heads per key head
    int head_blocks;  // blocks the group is cut into, of block_heads heads at most
    int block_heads;
    int capacity;     // tokens a row's table holds
    int wide;         // the keys (or values) span more than 2^32 chunks of 16 bytes
    int window, sinks;
    float scale_log2;  // scale * log2(e)
    uint16_t *out;     // [rows][q_heads][head_dim]
    float *lse;        // [rows][q_heads] or nullptr
    unsigned *counters;  // workspace (attention_plan.cuh): zero between calls
    float *partials;     // workspace: the slots
};
// In two forms for decode_attention_shared_prefix_bf16.
struct SharedAttentionArgs : AttentionArgs {
    float *part;               // the rows' own tokens alone: [rows][q_heads][head_dim] in place of out
    const int *prefix_table;   // joined: the prefix's pages,
    const int *prefix_length;  // its tokens,
    int prefix_capacity;       // and how many the table holds
};
cudaError_t launch_decode_attention(const AttentionArgs &a, int head_dim, int num_sms, int device,
                                    cudaStream_t stream, bool pdl);
cudaError_t attention_error_word(int **word);

// Attention over a prefix that all rows share (decode_attention_shared_prefix_bf16): the
// prefix's partials, the rows' own tokens in FP32, and the join (three launches, in this
// order; prefix_plan.cuh). Strides in elements.
struct PrefixArgs {
    const uint16_t *q;  // rows of q_heads * head_dim
    long long q_stride;
    const uint16_t *k, *v;
    int num_pages, page_size;
    int page_shift;  // log2(page_size), or -1
    long long page_stride, token_stride, head_stride;
    const int *table;   // [capacity / page_size]
    const int *length;  // one
    int capacity;       // tokens the table holds
    int rows, q_heads, kv_heads;
    int group;          // query heads per key head
    int tokens, blocks;  // PrefixPlan
    int lanes, ranges;   // blocks side by side, and the most ranges
    float scale_log2;
    int box_rows;       // tokens of a tensor map's box, or 0: no maps
    int head_chunks;    // prefix_merged: 128-byte chunks from head to head
    float *slots;       // workspace
    int slot_floats;
    const float *own_out, *own_lse;  // workspace: [rows][q_heads][head_dim] and [rows][q_heads]
    uint16_t *out;
    float *lse;  // or nullptr
    unsigned long long wait_limit_ns;
    int selftest;  // 1: an issuer of products waits on a barrier that nothing completes
};
// Tokens of a TMA box of the keys and values, all of one page, or 0 if boxes will not do (tiles
// must be whole boxes, and a box whole swizzle atoms).
int prefix_box_rows(int page_size, int tokens);
cudaError_t launch_prefix_attention(const CUtensorMap &k_map, const CUtensorMap &v_map, const PrefixArgs &a,
                                    int head_dim, int device, cudaStream_t stream, bool pdl);
cudaError_t launch_decode_attention_part(const SharedAttentionArgs &a, int head_dim, int num_sms, int device,
                                         cudaStream_t stream);
cudaError_t launch_decode_attention_joined(const SharedAttentionArgs &a, int head_dim, int num_sms, int device,
                                           cudaStream_t stream, bool pdl);
cudaError_t launch_prefix_join(const PrefixArgs &a, int head_dim, int num_sms, cudaStream_t stream);
cudaError_t prefix_error_word(int **word);
cudaError_t attention_part_error_word(int **word);
cudaError_t attention_joined_error_word(int **word);

// Log probabilities, entropy and top alternatives of rows of logits (token_logprobs_bf16).
constexpr int kLogprobMaxTop = 32;
struct LogprobArgs {
    const uint16_t *logits;
    long long stride;
    int M, V;
    const long long *tokens;  // [M][given]
    int given;
    float *logprobs;
    float *entropy, *lse;  // [M] or nullptr
    int top;
    float *top_logprobs;    // [M][top] or nullptr
    long long *top_tokens;  // [M][top] or nullptr
};
cudaError_t launch_token_logprobs(const LogprobArgs &a, int num_sms, cudaStream_t stream, bool pdl);
cudaError_t logprob_error_word(int **word);

}  // namespace skinny
