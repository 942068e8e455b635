// The C ABI's operators of a decode step that serves many requests (include/skinny.h):
// argument checks and launches. Every check runs before any launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "api_internal.h"
#include "kernels.h"
#include "prefix_plan.cuh"
#include "skinny.h"

using namespace skinny;

namespace {

struct Range {
    const void *p;
    size_t n;
};

// No output may overlap an input or another output. Absent ones are null.
template <int I, int O>
bool outputs_clear(const Range (&in)[I], const Range (&outs)[O]) {
    for (int i = 0; i < O; ++i) {
        if (!outs[i].p || !outs[i].n) continue;
        for (const Range &b : in)
            if (b.p && b.n && overlaps(outs[i].p, outs[i].n, b.p, b.n)) return false;
        for (int j = i + 1; j < O; ++j)
            if (outs[j].p && outs[j].n && overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return false;
    }
    return true;
}

// Whether the attention reads the prefix with every row's own tokens, in one launch, instead of
// reading it once and joining: `tokens` is what the prefix's table holds. Every row then reads the
// whole prefix, from L2 all but once, which is less than the time of two more launches and of the
// partial results of every row and head up to about 12 MiB and 20 KiB a row and head, for heads of
// up to 128: 12.2 against 14.7 us for 4 rows x 7 heads behind 509 tokens (1 MB), 14.3 against 15.2
// for 64 x 7 behind 500 (16 MB), 20.7 against 26.8 for 64 x 56 over 8 behind 200 (52 MB); but 17.5
// against 15.4 for 4 x 7 behind 8000 (16 MB), 20.6 against 15.2 for 64 x 7 behind 2000 (66 MB). With
// more than 8 heads to a key head that kernel takes longer and the tensor cores do not: 16 x 16 over
// 1 behind 500 (4 MB) 16.5 and 14.8, 64 x 32 over 2 behind 200 18.2 and 20.0; with more than 16 always (4 x 96 over 2
// behind 100 21.4 and 14.7).
// A single row's prefix is shared with nobody: 14.0 against 14.2 us for 7 heads behind 8000 tokens,
// 50.7 against 63.6 for 56 heads over 8 behind 60000. Wider heads run on the tensor cores from the
// first token on: 16.9 us for 8 rows x 16 heads of 256 behind 2000 tokens, 34.1 in one launch.
// (Times inside a graph.)
bool joined_is_faster(int rows, int q_heads, int kv_heads, int head_dim, long long tokens) {
    const int group = q_heads / kv_heads;
    if (head_dim > 128 || group > 16) return false;
    const long long bytes = tokens * rows * kv_heads * head_dim * 4, joins = rows * q_heads * (20ll << 10);
    if (group > 8) return bytes * group / 8 <= joins;
    return rows == 1 || bytes <= (12ll << 20) + joins;
}
long long attention_tiles(int rows, int kv_heads, int head_blocks, long long tokens) {
    return (tokens + kAttnMinTile - 1) / kAttnMinTile * rows * kv_heads * head_blocks;
}

template <int N>
int check_on_device(const Range (&all)[N], int dev) {
    for (const Range &b : all)
        if (b.p && b.n)
            if (int st = check_device_pointer(b.p, dev)) return st;
    return SKINNY_OK;
}

constexpr unsigned long long kWaitLimitNs = 1000000000ull;  // 1 s per wait of the prefix's kernel

int shared_prefix(const skinny_shared_prefix_attention_args *p, const skinny_launch_opts *opts, void *stream,
                  int selftest, unsigned long long limit_ns);

}  // namespace

extern "C" {

int token_logprobs_bf16(const skinny_token_logprobs_args *p, const skinny_launch_opts *opts, void *stream) {
    if (!p || !p->logits || (p->given > 0 && (!p->tokens || !p->logprobs))) return SKINNY_ERR_NULL;
    if (p->M < 1 || p->M > SKINNY_LOGPROBS_MAX_ROWS || p->V < 1 || p->V > (1 << 30) || p->given < 0 ||
        p->given > (1 << 20) || p->top < 0 || p->top > SKINNY_LOGPROBS_MAX_TOP || p->top > p->V ||
        p->logits_stride < p->V || p->logits_stride > (1ll << 32))
        return SKINNY_ERR_SHAPE;
    const bool lists = p->top > 0 && (p->top_logprobs || p->top_tokens);
    if (p->given == 0 && !p->entropy && !p->lse && !lists) return SKINNY_ERR_NULL;
    if (!aligned(p->logits, 2) || !aligned(p->entropy, 4) || !aligned(p->lse, 4) ||
        (p->given > 0 && (!aligned(p->tokens, 8) || !aligned(p->logprobs, 4))) ||
        (lists && (!aligned(p->top_logprobs, 4) || !aligned(p->top_tokens, 8))))
        return SKINNY_ERR_ALIGN;
    const size_t M = p->M, asked = M * p->given, listed = lists ? M * p->top : 0;
    const Range in[] = {{p->logits, row_span(p->M, p->logits_stride, p->V)}, {p->tokens, asked * 8}};
    const Range outs[] = {{p->logprobs, asked * 4}, {p->entropy, M * 4}, {p->lse, M * 4},
                          {p->top_logprobs, listed * 4}, {p->top_tokens, listed * 8}};
    if (!outputs_clear(in, outs)) return SKINNY_ERR_ALIAS;
    LaunchSettings ls;
    int st, dev;
    DeviceState *d = nullptr;
    if ((st = resolve_settings(opts, &ls)) || (st = current_device(&dev)) || (st = device_state(dev, &d)) ||
        (st = check_on_device(in, dev)) || (st = check_on_device(outs, dev)))
        return st;
    static_assert(kLogprobMaxTop == SKINNY_LOGPROBS_MAX_TOP, "the header's number");
    LogprobArgs a = {};
    a.logits = static_cast<const uint16_t *>(p->logits);
    a.stride = p->logits_stride;
    a.M = p->M;
    a.V = p->V;
    a.tokens = static_cast<const long long *>(p->tokens);
    a.given = p->given;
    a.logprobs = static_cast<float *>(p->logprobs);
    a.entropy = static_cast<float *>(p->entropy);
    a.lse = static_cast<float *>(p->lse);
    a.top = lists ? p->top : 0;
    a.top_logprobs = static_cast<float *>(p->top_logprobs);
    a.top_tokens = static_cast<long long *>(p->top_tokens);
    if (launch_token_logprobs(a, d->sms, static_cast<cudaStream_t>(stream), ls.pdl) != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

size_t skinny_shared_prefix_workspace_bytes(int rows, int q_heads, int kv_heads, int head_dim, int num_sms) {
    if (rows < 1 || rows > SKINNY_ATTENTION_MAX_ROWS || kv_heads < 1 || q_heads < 1 || q_heads > kMaxHeads ||
        q_heads % kv_heads != 0 || num_sms < 1 ||
        (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 192 && head_dim != 256))
        return 0;
    return prefix_workspace(rows, q_heads, kv_heads, head_dim, attn_sms(num_sms)).bytes;
}

int decode_attention_shared_prefix_bf16(const skinny_shared_prefix_attention_args *p,
                                        const skinny_launch_opts *opts, void *stream) {
    return shared_prefix(p, opts, stream, 0, kWaitLimitNs);
}

int skinny_shared_prefix_selftest(const skinny_shared_prefix_attention_args *p, long long timeout_ns, void *stream) {
    if (timeout_ns < 1000 || timeout_ns > 2000000000LL) return SKINNY_ERR_ARG;
    return shared_prefix(p, nullptr, stream, 1, static_cast<unsigned long long>(timeout_ns));
}

}  // extern "C"

namespace {

int shared_prefix(const skinny_shared_prefix_attention_args *p, const skinny_launch_opts *opts, void *stream,
                  int selftest, unsigned long long limit_ns) {
    if (!p || !p->prefix_table || !p->prefix_length) return SKINNY_ERR_NULL;
    // The rows' own tokens follow the rules of decode_attention_bf16.
    skinny_decode_attention_args own = {};
    own.q = p->q;
    own.q_stride = p->q_stride;
    own.rows = p->rows;
    own.q_heads = p->q_heads;
    own.cache = p->cache;
    own.block_table = p->block_table;
    own.table_stride = p->table_stride;
    own.table_width = p->table_width;
    own.lengths = p->lengths;
    own.scale = p->scale;
    own.out = p->out;
    own.lse = p->lse;
    own.workspace = p->workspace;
    own.workspace_bytes = p->workspace_bytes;
    size_t pool = 0;
    int st = check_attention(&own, &pool);
    if (st) return st;
    const skinny_kv_cache *c = &p->cache;
    const int D = c->head_dim, group = p->q_heads / c->kv_heads;
    const PrefixPlan plan = prefix_plan(p->rows, group, D);
    const long long capacity = static_cast<long long>(p->prefix_width) * c->page_size;
    if (p->prefix_width < 1 || capacity >= (1ll << 30) ||
        (capacity + 63) / 64 * c->kv_heads >= (1ll << 31))
        return SKINNY_ERR_SHAPE;
    if (!aligned(p->prefix_table, 4) || !aligned(p->prefix_length, 4)) return SKINNY_ERR_ALIGN;
    const size_t heads = static_cast<size_t>(p->rows) * p->q_heads;
    const Range in[] = {{p->q, row_span(p->rows, p->q_stride, static_cast<long long>(p->q_heads) * D)},
                        {c->k, pool}, {c->v, pool},
                        {p->prefix_table, static_cast<size_t>(p->prefix_width) * 4}, {p->prefix_length, 4},
                        {p->block_table, (static_cast<size_t>(p->rows - 1) * p->table_stride + p->table_width) * 4},
                        {p->lengths, static_cast<size_t>(p->rows) * 4}};
    const Range outs[] = {{p->out, heads * D * 2}, {p->lse, heads * 4}, {p->workspace, p->workspace_bytes}};
    if (!outputs_clear(in, outs)) return SKINNY_ERR_ALIAS;
    LaunchSettings ls;
    int dev;
    DeviceState *d = nullptr;
    if ((st = resolve_settings(opts, &ls)) || (st = current_device(&dev)) || (st = device_state(dev, &d))) return st;
    const int sms = attn_sms(d->sms);
    const PrefixWorkspace ws = prefix_workspace(p->rows, p->q_heads, c->kv_heads, D, sms);
    if (p->workspace_bytes < ws.bytes) return SKINNY_ERR_SHAPE;
    if ((st = check_on_device(in, dev)) || (st = check_on_device(outs, dev))) return st;
    char *base = static_cast<char *>(p->workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    SharedAttentionArgs o = {};
    attention_args(&own, pool, &o);
    // Both kinds of tokens are counted in one int there, and so are the tiles.
    const long long tokens = o.capacity + capacity;
    if (!selftest && joined_is_faster(p->rows, p->q_heads, c->kv_heads, D, capacity) && tokens < (1ll << 31) - kAttnMinTile &&
        attention_tiles(p->rows, c->kv_heads, o.head_blocks, tokens) < (1ll << 31)) {
        o.prefix_table = static_cast<const int *>(p->prefix_table);
        o.prefix_length = static_cast<const int *>(p->prefix_length);
        o.prefix_capacity = static_cast<int>(capacity);
        if (launch_decode_attention_joined(o, D, sms, dev, s, ls.pdl) != cudaSuccess) {
            cudaGetLastError();
            return SKINNY_ERR_LAUNCH;
        }
        return SKINNY_OK;
    }
    o.out = nullptr;
    o.part = reinterpret_cast<float *>(base + ws.own_out);
    o.lse = reinterpret_cast<float *>(base + ws.own_lse);
    PrefixArgs a = {};
    a.q = o.q;
    a.q_stride = o.q_stride;
    a.k = o.k;
    a.v = o.v;
    a.num_pages = o.num_pages;
    a.page_size = o.page_size;
    a.page_shift = o.page_shift;
    a.page_stride = o.page_stride;
    a.token_stride = o.token_stride;
    a.head_stride = o.head_stride;
    a.table = static_cast<const int *>(p->prefix_table);
    a.length = static_cast<const int *>(p->prefix_length);
    a.capacity = static_cast<int>(capacity);
    a.rows = p->rows;
    a.q_heads = p->q_heads;
    a.kv_heads = c->kv_heads;
    a.group = group;
    a.tokens = plan.tokens;
    a.blocks = plan.blocks;
    const int ctas = prefix_ctas(p->rows, c->kv_heads, D, plan, capacity, o.capacity, sms);
    a.lanes = prefix_lanes(plan.blocks, ctas);
    // No more ranges than the table could ever hold tiles.
    a.ranges = static_cast<int>(std::min<long long>(prefix_ranges(plan.blocks, ctas),
                                                    (capacity + plan.tokens - 1) / plan.tokens * c->kv_heads));
    a.scale_log2 = o.scale_log2;
    a.slots = reinterpret_cast<float *>(base + ws.slots);
    a.slot_floats = static_cast<int>(prefix_slot_floats(D, static_cast<long long>(p->rows) * group));
    a.own_out = o.part;
    a.own_lse = o.lse;
    a.out = static_cast<uint16_t *>(p->out);
    a.lse = static_cast<float *>(p->lse);
    a.wait_limit_ns = limit_ns;
    a.selftest = selftest;
    alignas(64) CUtensorMap k_map = {}, v_map = {};
    a.box_rows = prefix_box_rows(c->page_size, plan.tokens);
    a.head_chunks = static_cast<int>(std::min<long long>(c->head_stride / 64, 1ll << 30));
    if (a.box_rows > 0 && !(encode_cache_map(&k_map, c->k, c, a.box_rows, prefix_merged(D)) &&
                            encode_cache_map(&v_map, c->v, c, a.box_rows, prefix_merged(D))))
        a.box_rows = 0;
    if (launch_prefix_attention(k_map, v_map, a, D, dev, s, ls.pdl) != cudaSuccess ||
        launch_decode_attention_part(o, D, ctas < sms ? sms - a.ranges * a.lanes : sms, dev, s) != cudaSuccess ||
        launch_prefix_join(a, D, sms, s) != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

}  // namespace
