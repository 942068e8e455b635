// The C ABI's operators of a decode step that serves many requests (include/skinny.h):
// argument checks and launches. Every check runs before any launch.
#include <cuda_runtime.h>

#include <cmath>

#include "api_internal.h"
#include "kernels.h"
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

template <int N>
int check_on_device(const Range (&all)[N], int dev) {
    for (const Range &b : all)
        if (b.p && b.n)
            if (int st = check_device_pointer(b.p, dev)) return st;
    return SKINNY_OK;
}

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

}  // extern "C"
