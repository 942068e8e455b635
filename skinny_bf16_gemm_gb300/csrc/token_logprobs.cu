// Log probabilities of given tokens, entropy and top alternatives of rows of logits on
// GB300 (sm_103a).
//
//   m = max x_j,  S = sum exp(x_j - m),  lse = m + log S
//   logprob(t) = (x_t - m) - log S,  entropy = log S - sum exp(x_j - m)(x_j - m) / S
// and the `top` largest logits, of equal ones the lower index first. One pass over the row
// with the running maximum and both sums; bound by HBM (2 bytes a logit).
//
// A row is one cluster of C CTAs (C = 1: one CTA) whose threads take its 16-byte vectors in
// turn; the CTAs' maxima, sums and top lists meet in the first one's shared memory, so there
// is no workspace and nothing to reset. A row may start at any 2-byte address: the values
// before its first and after its last whole vector are single loads.
//
// The top list needs no second pass over the row: the `top`-th largest of the threads' own
// maxima bounds the `top`-th largest value from below (that many threads have a value as
// large), so only those threads' values are read again, of most of them no more than the
// kUnroll vectors with their maximum: a thread keeps the largest of its other rounds, too.
// What reaches the bound is listed and ranked by (value, index).
// Where ties at the bound or few heavy threads overflow the list, the exact bound is found by
// bisecting the 16-bit values and the ties are taken in the order of their index.
//
// Measured (in a graph): 2048 rows of 163840 120.4 us, 5.6 TB/s (109.0, 6.2 TB/s, without the
// list of 8); 64 rows of 163840, on 8 CTAs each, 9.2 us without a list and 15.7 with one of 20:
// bisecting the bound over the threads' maxima by one warp, reading the flagged rounds again and the join
// of 8 lists are three latencies one after another. 6.5 us for one row of 20480.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace skinny {
namespace {

constexpr int kUnroll = 4;     // vectors a thread has on their way
constexpr int kList = 1024;    // candidates (and as many ties) that are ranked at once
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.44269504088896341f;
// The maximum of no logits: finite, so that -inf minus it is -inf.
constexpr float kNoMaximum = -3.402823466e+38f;
// Below this exponent a weight is 0; the product with it must not be 0 * -inf.
constexpr float kFloor = -1e4f;
__device__ int g_logprob_err;  // nonzero: a token index was out of range

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A whole number in the logits' order, from -inf (0x7F) up. -0 is +0, NaN counts as -inf.
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
    if ((bits & 0x7FFFu) > 0x7F80u) bits = 0xFF80u;
    if (bits == 0x8000u) bits = 0u;
    return (bits & 0x8000u) ? 0xFFFFu - bits : bits | 0x8000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(((key & 0x8000u) ? key & 0x7FFFu : 0xFFFFu - key) << 16);
}
__device__ __forceinline__ float logit_of(uint32_t bits) { return __uint_as_float(bits << 16); }

// Running maximum, sum of exp(x - m) and sum of exp(x - m) (x - m).
struct Sums {
    float m, s1, s2;
};
__device__ __forceinline__ void raise(Sums &a, float m) {
    const float d = fmaxf(a.m - m, kFloor), f = exp2_approx(d * kLog2e);
    a.s2 = f * (a.s2 + a.s1 * d);
    a.s1 *= f;
    a.m = m;
}
__device__ __forceinline__ void add(Sums &a, Sums b) {
    const float m = fmaxf(a.m, b.m);
    raise(a, m);
    raise(b, m);
    a.s1 += b.s1;
    a.s2 += b.s2;
}

__device__ __forceinline__ uint4 load_vector(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t bits_at(const uint4 &v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return (e & 1) ? w >> 16 : w & 0xFFFFu;
}

template <int C, int kThreads>
__global__ void __launch_bounds__(kThreads, 1280 / kThreads) token_logprobs_kernel(const LogprobArgs a) {
    constexpr int kWarps = kThreads / 32;
    __shared__ Sums sm_sums[kWarps];
    __shared__ Sums sm_peers[C];
    __shared__ unsigned long long sm_tops[C * kLogprobMaxTop];
    __shared__ unsigned long long sm_list[kList], sm_ties[kList];
    __shared__ int sm_counts[2];
    __shared__ int sm_scan[kWarps];
    __shared__ uint32_t sm_bound;
    __shared__ uint16_t sm_maxima[kThreads];
    __shared__ int sm_again[kWarps][32];  // what a warp reads again: vectors, then lanes
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int rank = C > 1 ? static_cast<int>(blockIdx.x % C) : 0;
    const long long row = blockIdx.x / C;
    const uint16_t *x = a.logits + row * a.stride;
    const int top = a.top;

    // Whole vectors [v_begin, v_end) of this CTA; the first value of vector v is head + 8 v.
    const int before = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / 2;
    const int head = before < a.V ? before : a.V;
    const int vectors = (a.V - head) / 8, tail = a.V - head - vectors * 8;
    const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
    const int v_begin = static_cast<int>(static_cast<long long>(vectors) * rank / C);
    const int v_end = static_cast<int>(static_cast<long long>(vectors) * (rank + 1) / C);
    // This thread's single value before or after the vectors, or -1.
    const int lone = rank == 0 && tid < head ? tid : -1;
    const int late = rank == C - 1 && tid < tail ? a.V - tail + tid : -1;

    ptx::pdl_launch_dependents();
    ptx::pdl_wait();

    // ---- one pass: maximum and sums ----
    Sums sums = {kNoMaximum, 0.0f, 0.0f};
    float best = -INFINITY;    // this thread's largest value
    float second = -INFINITY;  // the largest of its other rounds
    int best_at = v_end;       // the first vector of the round with the largest
    auto take = [&](float v) {  // as another round's
        second = fmaxf(second, v);
        if (v > sums.m) raise(sums, v);
        const float t = v - sums.m, e = exp2_approx(t * kLog2e);
        sums.s1 += e;
        sums.s2 += e * fmaxf(t, kFloor);
    };
    if (lone >= 0) take(logit_of(x[lone]));
    if (late >= 0) take(logit_of(x[late]));
    for (int v = v_begin + tid; v < v_end; v += kThreads * kUnroll) {
        uint4 w[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            w[u] = v + u * kThreads < v_end ? load_vector(xv + v + u * kThreads)
                                            : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
        float most = -INFINITY;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, logit_of(bits_at(w[u], e)));
        if (most > best) {
            second = fmaxf(second, best);
            best = most;
            best_at = v;
        } else {
            second = fmaxf(second, most);
        }
        if (most > sums.m) raise(sums, most);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = logit_of(bits_at(w[u], e)) - sums.m, p = exp2_approx(t * kLog2e);
                sums.s1 += p;
                sums.s2 += p * fmaxf(t, kFloor);
            }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        add(sums, {__shfl_xor_sync(0xFFFFFFFFu, sums.m, o), __shfl_xor_sync(0xFFFFFFFFu, sums.s1, o),
                   __shfl_xor_sync(0xFFFFFFFFu, sums.s2, o)});
    if (lane == 0) sm_sums[warp] = sums;
    if (tid < 2) sm_counts[tid] = 0;
    __syncthreads();

    // ---- this CTA's top list ----
    if (top > 0) {
        const uint32_t mine = key_of(__float_as_uint(fmaxf(best, second)) >> 16);
        // The top-th largest of the threads' maxima, bit by bit, by one warp with kWarps of them a
        // lane (0: fewer threads than that).
        sm_maxima[tid] = static_cast<uint16_t>(mine);
        __syncthreads();
        if (warp == 0) {
            uint32_t k[kWarps], found = 0;
#pragma unroll
            for (int e = 0; e < kWarps; ++e) k[e] = sm_maxima[e * 32 + lane];
#pragma unroll 1
            for (uint32_t bit = 0x8000u; bit != 0; bit >>= 1) {
                int n = 0;
#pragma unroll
                for (int e = 0; e < kWarps; ++e) n += k[e] >= (found | bit);
                if (__reduce_add_sync(0xFFFFFFFFu, n) >= top) found |= bit;
            }
            if (lane == 0) sm_bound = found;
        }
        __syncthreads();
        uint32_t bound = sm_bound;

        // Every value of this thread in turn.
        auto each = [&](auto &&f) {
            if (lone >= 0) f(key_of(x[lone]), lone);
            for (int v = v_begin + tid; v < v_end; v += kThreads) {
                const uint4 w = load_vector(xv + v);
                for (int e = 0; e < 8; ++e) f(key_of(bits_at(w, e)), head + v * 8 + e);
            }
            if (late >= 0) f(key_of(x[late]), late);
        };
        auto entry = [](uint32_t key, int i) {
            return static_cast<unsigned long long>(key) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(i));
        };
        // List a value: those above the bound, and up to kList of the ties with it.
        auto put = [&](uint32_t key, int i) {
            if (key < bound) return;
            if (key > bound) {
                const int at = atomicAdd(&sm_counts[0], 1);
                if (at < kList) sm_list[at] = entry(key, i);
            } else if (*static_cast<volatile int *>(&sm_counts[1]) <= kList) {
                const int at = atomicAdd(&sm_counts[1], 1);
                if (at < kList) sm_ties[at] = entry(key, i);
            }
        };
        // The values of the threads that reach the bound, their vectors dealt to the lanes of their
        // warp: the round with the largest value, or all if another reaches the bound too.
        const bool many = key_of(__float_as_uint(second) >> 16) >= bound, one = mine >= bound && !many;
        if (many) {
            if (lone >= 0) put(key_of(x[lone]), lone);
            if (late >= 0) put(key_of(x[late]), late);
        }
        const unsigned ones = __ballot_sync(0xFFFFFFFFu, one), all = __ballot_sync(0xFFFFFFFFu, many);
        const unsigned below = (1u << lane) - 1u;
        if (one) sm_again[warp][__popc(ones & below)] = best_at;
        if (many) sm_again[warp][__popc(ones) + __popc(all & below)] = v_begin + tid;
        __syncwarp();
        const int each_has = (v_end - v_begin + kThreads - 1) / kThreads, first = __popc(ones) * kUnroll;
        for (int item = lane; item < first + __popc(all) * each_has; item += 32) {
            int who = item / kUnroll, i = item % kUnroll;
            if (item >= first) {
                who = (item - first) / each_has;
                i = item - first - who * each_has;
                who += __popc(ones);
            }
            const int v = sm_again[warp][who] + i * kThreads;
            if (v >= v_end) continue;
            const uint4 w = load_vector(xv + v);
#pragma unroll
            for (int e = 0; e < 8; ++e) put(key_of(bits_at(w, e)), head + v * 8 + e);
        }
        __syncthreads();
        if (sm_counts[0] > kList) {
            // Few threads with very many large values: bisect for the exact bound.
            uint32_t lo = bound, hi = 0x10000u;
            while (hi - lo > 1) {
                const uint32_t mid = (lo + hi) / 2;
                int n = 0;
                if (mine >= mid) each([&](uint32_t key, int) { n += key >= mid; });
                n = __reduce_add_sync(0xFFFFFFFFu, n);
                __syncthreads();
                if (lane == 0) sm_scan[warp] = n;
                __syncthreads();
                n = 0;
                for (int w = 0; w < kWarps; ++w) n += sm_scan[w];
                if (n >= top) lo = mid; else hi = mid;
            }
            bound = lo;
            __syncthreads();
            if (tid < 2) sm_counts[tid] = 0;
            __syncthreads();
            if (mine >= bound) each(put);
            __syncthreads();
        }
        const int above = sm_counts[0];
        int ties = sm_counts[1];
        if (ties > kList && above < top) {
            // More ties than are listed: the ones of lowest index, vector by vector.
            const int need = top - above;
            int have = 0;
            auto take_ties = [&](int n, auto &&index) {  // this thread's n ties of a stretch
                int at = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xFFFFFFFFu, at, o);
                    if (lane >= o) at += up;
                }
                __syncthreads();
                if (lane == 31) sm_scan[warp] = at;
                __syncthreads();
                int all = 0;
                for (int w = 0; w < kWarps; ++w) {
                    if (w < warp) at += sm_scan[w];
                    all += sm_scan[w];
                }
                at += have - n;
                for (int i = 0; i < n && at < need; ++i, ++at) sm_ties[at] = entry(bound, index(i));
                have += all;
            };
            take_ties(lone >= 0 && key_of(x[lone]) == bound, [&](int) { return lone; });
            for (int v0 = v_begin; v0 < v_end && have < need; v0 += kThreads) {
                const int v = v0 + tid;
                unsigned at = 0;  // which of the vector's values are ties
                if (v < v_end) {
                    const uint4 w = load_vector(xv + v);
                    for (int e = 0; e < 8; ++e) at |= static_cast<unsigned>(key_of(bits_at(w, e)) == bound) << e;
                }
                take_ties(__popc(at), [&](int) {
                    const int e = __ffs(at) - 1;
                    at &= at - 1;
                    return head + v * 8 + e;
                });
            }
            if (have < need) take_ties(late >= 0 && key_of(x[late]) == bound, [&](int) { return late; });
            ties = have < need ? have : need;
            __syncthreads();
        }
        // Rank the listed values; the place of a list in the first CTA's shared memory.
        const int n = above + (above < top ? ties : 0);
        uint32_t to = ptx::smem_addr(sm_tops + rank * kLogprobMaxTop);
        if constexpr (C > 1) to = ptx::map_to_cluster_rank(to, 0);
        auto listed = [&](int i) { return i < above ? sm_list[i] : sm_ties[i - above]; };
        auto larger = [](const unsigned long long *list, int count, unsigned long long e) {
            int better = 0;
#pragma unroll 8
            for (int j = 0; j < count; ++j) better += list[j] > e;
            return better;
        };
        if constexpr (C > 1) {
            __syncthreads();
            ptx::cluster_sync();  // the first CTA runs: its memory may be written
        }
        for (int i = tid; i < n; i += kThreads) {
            const unsigned long long e = listed(i);
            const int better = larger(sm_list, above, e) + larger(sm_ties, n - above, e);
            if (better < top) ptx::st_cluster_u64(to + better * 8, e);
        }
        for (int i = n + tid; i < top; i += kThreads) ptx::st_cluster_u64(to + i * 8, 0ull);
    } else if constexpr (C > 1) {
        ptx::cluster_sync();
    }

    // ---- join ----
    if (tid == 0) {
        Sums s = sm_sums[0];
        for (int w = 1; w < kWarps; ++w) add(s, sm_sums[w]);
        uint32_t to = ptx::smem_addr(sm_peers + rank);
        if constexpr (C > 1) to = ptx::map_to_cluster_rank(to, 0);
        ptx::st_cluster_f32(to, s.m);
        ptx::st_cluster_f32(to + 4, s.s1);
        ptx::st_cluster_f32(to + 8, s.s2);
    }
    __syncthreads();
    if constexpr (C > 1) ptx::cluster_sync();
    if (rank != 0) return;
    Sums all = sm_peers[0];
#pragma unroll
    for (int c = 1; c < C; ++c) add(all, sm_peers[c]);
    const float log_sum = logf(all.s1);
    if (tid == 0) {
        if (a.lse != nullptr) a.lse[row] = all.m + log_sum;
        if (a.entropy != nullptr) a.entropy[row] = log_sum - __fdiv_rn(all.s2, all.s1);
    }
    for (int i = tid; i < a.given; i += kThreads) {
        const long long t = a.tokens[row * a.given + i];
        float p = 0.0f;  // a position that is not asked for
        if (t >= a.V) {
            atomicOr(&g_logprob_err, 1);
            p = NAN;
        } else if (t >= 0) {
            p = (logit_of(x[t]) - all.m) - log_sum;
        }
        a.logprobs[row * a.given + i] = p;
    }
    for (int i = tid; i < C * top; i += kThreads) {
        const unsigned long long e = sm_tops[i / top * kLogprobMaxTop + i % top];
        if (e == 0) continue;
        int better = C > 1 ? 0 : i;
        if constexpr (C > 1)
            for (int c = 0; c < C; ++c)
#pragma unroll 8
                for (int j = 0; j < top; ++j) better += sm_tops[c * kLogprobMaxTop + j] > e;
        if (better >= top) continue;
        const float v = value_of(static_cast<uint32_t>(e >> 32));
        if (a.top_logprobs != nullptr) a.top_logprobs[row * top + better] = (v - all.m) - log_sum;
        if (a.top_tokens != nullptr)
            a.top_tokens[row * top + better] = static_cast<long long>(0xFFFFFFFFu - static_cast<uint32_t>(e));
    }
}

template <int C, int kThreads>
cudaError_t launch_threads(const LogprobArgs &a, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.M) * C, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<C, kThreads>, a);
}
template <int C>
cudaError_t launch(const LogprobArgs &a, int threads, cudaStream_t stream, bool pdl) {
    return threads == 256 ? launch_threads<C, 256>(a, stream, pdl) : launch_threads<C, 128>(a, stream, pdl);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs &a, int num_sms, cudaStream_t stream, bool pdl) {
    // CTAs a row: as many as keep every SM's threads on a row, but no fewer than a vector a
    // thread.
    const int vectors = a.V / 8;
    int c = kMaxCluster;
    while (c > 1 && (vectors < c * 128 || static_cast<long long>(a.M) * c > 8ll * num_sms)) c /= 2;
    // 128 threads: twice the rows an SM, so that one's list is made while others are read (512 rows
    // of 32000, list of 8: 14.7 us, 20.1 with 256; 4096 of 50257: 91.5, 95.0; 128 of 163840, on 8
    // CTAs: 17.3, 22.2). 256 where a CTA's part is long and all CTAs run at once anyway (64 rows of
    // 163840: 15.7, 17.1; one: 9.9, 12.6), or where the last CTAs of long rows would run with much
    // of the GPU idle (2048 of 100000: 84, 88; of 163840: 120, 131).
    const long long ctas = static_cast<long long>(a.M) * c, at_once = 5ll * num_sms;
    auto filled = [&](long long places) { return static_cast<double>(ctas) / ((ctas + places - 1) / places * places); };
    const int threads = ctas <= at_once ? (vectors / c >= 2048 ? 256 : 128)
                                        : (a.V >= 80000 && filled(at_once) > 1.15 * filled(2 * at_once) ? 256 : 128);
    if (c == 8) return launch<8>(a, threads, stream, pdl);
    if (c == 4) return launch<4>(a, threads, stream, pdl);
    if (c == 2) return launch<2>(a, threads, stream, pdl);
    return launch<1>(a, threads, stream, pdl);
}

cudaError_t logprob_error_word(int **word) { return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_logprob_err); }

}  // namespace skinny
