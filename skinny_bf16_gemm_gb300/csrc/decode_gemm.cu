// Decode GEMM for GB300 (sm_103a): out[M, N] = x[M, K] @ W[N, K]^T, BF16 operands,
// FP32 accumulation, one BF16 rounding ("drafter/linears": module text and
// DraftGemm). M <= 64, so the time is the weight stream: every byte of W is read
// once from HBM by TMA and fed to the tensor cores while it is on chip.
//
// Persistent CTAs of 192 threads in three roles:
//   warp 0      TMA producer: W tiles [128 rows x 64 K] and x slices [MP x 64 K]
//               into a ring of STAGES shared-memory stages (128-byte swizzle);
//   warp 1      MMA issuer: tcgen05.mma kind::f16, M = 128 weight rows, N = MP
//               (x rows padded to 16, 32 or 64; the padding rows are TMA zero
//               fill), accumulating in tensor memory (two accumulator buffers);
//   warps 2..5  epilogue: tcgen05.ld of the accumulator (TMEM lane = weight row =
//               output column n, column = output row m), one BF16 rounding and
//               the store (for whole tiles of 32/64 padded rows through the
//               idle ring, as 16-byte row pieces), or the split-K fix-up.
// Work split (plan.cuh): one whole 128-row tile per CTA when the tiles nearly fill
// the GPU, otherwise the ceil(N/128) x ceil(K/64) weight blocks dealt to one CTA
// per SM as equal contiguous ranges (stream-K). A tile whose K range is shared
// by several CTAs is finished by the CTA holding its first K blocks (for which it
// is the last piece): the others publish their FP32 partials behind a release
// flag, and the finisher adds them in K order, so the bits do not depend on
// timing. Ranges go to CTAs in reverse block order, so a finisher waits only on
// CTAs with lower block indices, which the GPU dispatched before it.
// Ring depth (plan.cuh use_shallow_ring): the deep ring, one CTA per SM, for
// long streams; the shallow ring for short ones under programmatic dependent
// launch, so that the next kernel's CTA shares the SM. Before waiting on the
// previous kernel in the stream the producer already streams the first STAGES
// weight tiles and prefetches more into L2 -- behind decode_gemm_bf16_reduce_rmsnorm
// optionally more again once that call's reduce has seen its GEMM complete:
// weights never depend on the previous kernel, x may.
// Every wait is bounded (wait_limit_ns); a role that gives up records a bit in
// the device error word, the CTA drains its in-flight copies and MMAs, frees its
// tensor memory and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>
#include <type_traits>

#include "epilogue.cuh"
#include "kernels.h"
#include "plan.cuh"
#include "ptx.cuh"

namespace skinny {
namespace {

constexpr int kThreads = 192;
constexpr int kEpilogueThreads = 128;
constexpr int kWBytes = kBlockN * kBlockK * 2;
constexpr uint64_t kDrainLimitNs = 200000000ull;  // 0.2 s for copies already issued
// Weight blocks prefetched to L2, beyond the ring's first fill, before waiting
// on the previous kernel: 8 with the shallow ring, the caller's GemmArgs::l2_lead
// with the deep ring. Both short: the early requests share the SM and HBM with
// the previous kernel's last CTAs and slow them. Measured on GB300 for the
// shallow ring (its co-resident CTA is the previous kernel's): leads of 8-10
// beat 26 (most of a short range) by up to 1.4 us at N = 4096 and 3.5 us at
// N = 6144-7168 (K = 7168, 0.4-0.7 MB per CTA); 0-4 are slower again.
constexpr int kL2PrefetchShallow = 8;
// The longest a producer waits for the previous GEMM's completion signal before
// it goes on without the prefetch that depends on it (GemmArgs::l2_after_reduce).
constexpr uint64_t kAfterReduceWaitNs = 50000ull;
constexpr int kMaxShallowStages = 6;  // shallow rings have 5..6 stages, deep ones 9..11

// MP: padded row count (MMA N). STAGES: shared-memory ring depth. The deep ring
// (185-227 KB) keeps the most bytes in flight; the shallow one (~100-112 KB) lets
// the next kernel's CTAs be resident on the same SM while this one finishes, so
// with programmatic dependent launch they stream weights across the boundary
// (plan.cuh use_shallow_ring picks one by the weight bytes per CTA).
// LORA: how the adapters' part of a tile is worked out (decode_gemm_bf16_lora), see the kernel.
enum Lora { kNoLora, kLoraDirect, kLoraCopied };
constexpr int kLoraCopiedFrom = 24;  // the smallest rank that may go by kLoraCopied
template <int MP, int STAGES, int LORA = kNoLora>
struct Layout {
    static constexpr int kStages = STAGES;
    static constexpr int kAccCols = MP == 64 ? 64 : 32;  // TMEM columns per accumulator
    // Two accumulator buffers; LORA: the adapters' part of a tile, in the columns after them
    // (a power of two of columns in all).
    static constexpr int kTmemCols = (LORA ? 4 : 2) * kAccCols;
    static constexpr int kLoraCol = 2 * kAccCols;
    static constexpr int kXBytes = MP * kBlockK * 2;
    static constexpr int kStageBytes = kWBytes + kXBytes;
    static constexpr int kBarOffset = kStages * kStageBytes;
    static constexpr int kNumBars = 2 * kStages + 7;
    static constexpr int kRingBytes = kStages * kStageBytes;
    static constexpr int kMiscOffset = kBarOffset + kNumBars * 8;
    // LORA: the rows' adapters and their scales, then scale A x [M][rank] (as many bytes as the
    // call needs). Copied: before them the adapters in use and their rows, behind them the
    // epilogue warps' rings of rows of B, in what is left of kLoraBytes (at least 32 rows of rank
    // 128 a warp).
    static constexpr int kLoraOffset = kMiscOffset + 24, kLoraListOffset = kLoraOffset + 2 * kMaxM * 4;
    static constexpr int kLoraAxOffset = kLoraListOffset + (LORA == kLoraCopied ? 12 * kMaxM + 16 : 0);
    static constexpr int kLoraBytes = LORA == kLoraCopied ? 49152 + MP * kLoraMaxRank * 4 : 0;
    static constexpr int kBytes = LORA ? kLoraAxOffset + kLoraBytes : kMiscOffset + 16;
    static constexpr int kDynamicBytes = kBytes + 1024;  // slack to align the base to 1024
    static_assert(!LORA || kLoraOffset % 16 == 0, "16-byte loads of A x");
    static_assert(kStageBytes % 1024 == 0, "stages must keep 1024-byte alignment");
};

enum WaitResult { kWaitDone = 1, kWaitTimeout = 0, kWaitAborted = -1 };

// Wait for completion of the barrier phase with `parity`, giving up after
// limit_ns or as soon as another role of this CTA has aborted.
__device__ __forceinline__ int bounded_wait(uint32_t bar, uint32_t parity,
                                            const volatile uint32_t *abort_flag,
                                            uint64_t limit_ns) {
    if (ptx::mbar_try_wait(bar, parity)) return kWaitDone;
    const uint64_t t0 = ptx::global_timer_ns();
    for (uint32_t spin = 1;; ++spin) {
        if (ptx::mbar_try_wait(bar, parity)) return kWaitDone;
        if ((spin & 15u) == 0) {
            if (*abort_flag) return kWaitAborted;
            if (ptx::global_timer_ns() - t0 > limit_ns) return kWaitTimeout;
        }
    }
}

// Record a problem: the bit in the device error word, and a nonzero word in the
// caller's host-mapped memory when there is one (the host reads it without
// synchronising, so the library's next call can report it).
__device__ __forceinline__ void record_error(const GemmArgs &a, int bit) {
    atomicOr(a.err, bit);
    if (a.host_err != nullptr) {
        *reinterpret_cast<volatile int *>(a.host_err) = 1;
        __threadfence_system();
    }
}

__device__ __forceinline__ void raise_error(const GemmArgs &a, volatile uint32_t *abort_flag,
                                            int bit) {
    record_error(a, bit);
    *abort_flag = 1u;
}

// Barrier-wide OR of a predicate over the epilogue's 128 threads (named barrier 1).
__device__ __forceinline__ bool epilogue_any(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\t"
        "setp.ne.u32 a, %1, 0;\n\t"
        "bar.red.or.pred b, 1, 128, a;\n\t"
        "selp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(p))
        : "memory");
    return r != 0;
}

__device__ __forceinline__ uint16_t to_bf16_bits(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// The value an output element is rounded from: the FP32 sum itself, or for the
// lm_head logits ("drafter/linears", draft_logits) the soft-capped, scaled sum.
__device__ __forceinline__ float output_value(float v, const GemmArgs &a) {
    if (!a.logits) return v;
    if (a.soft_cap > 0.0f) v = __fmul_rn(tanhf(__fdiv_rn(v, a.soft_cap)), a.soft_cap);
    return __fmul_rn(v, a.scale);
}

// Store rows 0..M-1 of one tile's output (this thread's column n = tile * 128 +
// row; v[m] the values to round) through the idle ring: each thread puts its
// BF16 values in shared memory, then the 128 epilogue threads write 16-byte
// pieces of whole rows instead of one 2-byte store per row and thread. Needs
// 16-byte aligned rows (N a multiple of 8) and a ring nothing uses any more.
// Measured on GB300 for whole tiles of 32 and 64 padded rows with the deep
// ring: 0.3-0.6 us faster per call at N = 18432; no gain for 16 rows or on
// split tiles, and 0.2 us slower with the shallow ring, so only there.
template <int MP>
__device__ __forceinline__ void store_tile_staged(const float (&v)[MP], uint16_t *out, int M, int N,
                                                  int tile, int row, int etid, uint32_t stage) {
#pragma unroll
    for (int m = 0; m < MP; ++m)
        if (m < M)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage + (m * kBlockN + row) * 2),
                         "h"(to_bf16_bits(v[m])) : "memory");
    ptx::named_barrier_sync(1, kEpilogueThreads);
    const int pieces = M * (kBlockN / 8);
    for (int i = etid; i < pieces; i += kEpilogueThreads) {
        const int m = i / (kBlockN / 8), c = i % (kBlockN / 8);
        const int n0 = tile * kBlockN + c * 8;
        if (n0 < N) {
            uint4 w;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(stage + (m * kBlockN + c * 8) * 2) : "memory");
            *reinterpret_cast<uint4 *>(out + static_cast<size_t>(m) * N + n0) = w;
        }
    }
}

// Eight products of B and A x added to a row's two sums, of the even and the odd ones: one order for
// both forms of LORA below, so that a call's bits do not depend on which of them it goes by.
__device__ __forceinline__ void lora_add(float (&v)[2], const uint4 &b, const float4 &t0, const float4 &t1) {
    v[0] = fmaf(t0.x, __uint_as_float(b.x << 16), v[0]);
    v[1] = fmaf(t0.y, __uint_as_float(b.x & 0xFFFF0000u), v[1]);
    v[0] = fmaf(t0.z, __uint_as_float(b.y << 16), v[0]);
    v[1] = fmaf(t0.w, __uint_as_float(b.y & 0xFFFF0000u), v[1]);
    v[0] = fmaf(t1.x, __uint_as_float(b.z << 16), v[0]);
    v[1] = fmaf(t1.y, __uint_as_float(b.z & 0xFFFF0000u), v[1]);
    v[0] = fmaf(t1.z, __uint_as_float(b.w << 16), v[0]);
    v[1] = fmaf(t1.w, __uint_as_float(b.w & 0xFFFF0000u), v[1]);
}

// EPI: the epilogue of epilogue.cuh. LORA (with EPI): the adapters' second half,
// scale B_a (A_a x), a the row's adapter. Templates so that the plain kernel keeps its
// registers.
//
// LORA: the kernel is launched behind lora_shrink_kernel, which lets it start once x is
// there, so nothing but the epilogue waits for that kernel. While a tile's weights stream the
// epilogue's threads, idle otherwise, work its part out: thread = output column n, which multiplies
// row n of every B in use with A x of the adapter's rows, from shared memory, in FP32; the result
// waits in tensor memory. A tile's contributors (split K) share the work out. Two forms, by
// the call's rank and rows:
//   direct  each row of x takes its row of B to registers, eight rows at a time (those that share
//           an adapter find it in L2). For small ranks, whose 32 rows of a warp are few lines.
//   copied  each B in use once: the warp copies its 32 rows, one stretch of B, to shared memory
//           (cp.async, some adapters ahead, waited for by the warp alone), in the place of two or
//           three stages. From rank 64 on a load of 32 rows' pieces is 32 requests: 64 x 4096 x
//           4096 with 16 adapters of rank 128 50 us, direct 74; 32 x 18432 x 7168 with 8 of rank 64
//           54 and 65; but 64 x 7168 x 18432 with 64 of rank 16 65 and 62, 5 x 4099 x 1000 with 3 of
//           rank 8 13.6 and 11.1. From rank 24 on where a pool of so few adapters (how many of
//           them are in use only the device knows) serves so many rows that rank x rows is
//           96 x adapters or more: 64 x 18432 x 7168 with 32 of rank 48 63, direct 78;
//           49 x 2173 x 64 with 6 of rank 24 17.5 and 23.0; but 36 x 8521 x 288 with 19 of rank 32
//           24.5 and 23.4.
template <int MP, int STAGES, bool EPI, int LORA>
__global__ void __launch_bounds__(kThreads, 1)
    decode_gemm_kernel(const __grid_constant__ CUtensorMap w_map,
                       const __grid_constant__ CUtensorMap x_map, const GemmArgs args) {
    using L = Layout<MP, STAGES, LORA>;
    constexpr int S = L::kStages;
    constexpr bool kCopied = LORA == kLoraCopied;
    constexpr bool kShallow = STAGES <= kMaxShallowStages && !kCopied;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = ptx::smem_addr(smem);
    const uint32_t bar_full = sbase + L::kBarOffset;   // + 8 s
    const uint32_t bar_empty = bar_full + 8 * S;       // + 8 s
    const uint32_t bar_acc_full = bar_empty + 8 * S;   // + 8 b
    const uint32_t bar_acc_empty = bar_acc_full + 16;  // + 8 b
    const uint32_t bar_drain = bar_acc_empty + 16;
    const uint32_t bar_never = bar_drain + 8;
    const uint32_t bar_fix = bar_never + 8;             // split-K fix-up bulk copies
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + L::kMiscOffset);
    // misc[0]: tensor-memory base, misc[1]: abort flag

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const GemmGeometry g = make_geometry(args.M, args.N, args.K, gridDim.x);
    // This CTA's range of weight blocks (plan.cuh: reverse block order, so the
    // split-K finisher below waits only on CTAs with lower block indices).
    const int cta = range_of_block(g, static_cast<int>(blockIdx.x));
    const uint64_t limit = args.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar_acc_full + 8 * b, 1);
            ptx::mbar_init(bar_acc_empty + 8 * b, kEpilogueThreads);
        }
        ptx::mbar_init(bar_drain, 1);
        ptx::mbar_init(bar_never, 1);
        ptx::mbar_init(bar_fix, 1);
        misc[1] = 0u;
        ptx::fence_barrier_init();
    }
    if (warp == 0) {
        ptx::tmem_alloc(sbase + L::kMiscOffset, L::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = misc[0];
    volatile uint32_t *abort_flag = misc + 1;

    // The next kernel in the stream may launch now: its CTAs take SMs as they
    // free up (beside this one with the shallow ring), set up and stream their
    // first weights while this grid runs, and wait for it before touching
    // anything it writes.
    ptx::pdl_launch_dependents();

    // This CTA's blocks [b0, b1). Block indices stay below 2^31 (the host rejects
    // larger problems), so after the two 64-bit divisions of the range ends all
    // the plan arithmetic here is 32-bit.
    const long long b0 = cta_begin(g, cta);
    const long long b1 = cta_begin(g, cta + 1);
    const int total = static_cast<int>(b1 - b0);
    const BlockCursor start = {static_cast<int>(b0) / g.kblocks,
                               static_cast<int>(b0) - (static_cast<int>(b0) / g.kblocks) * g.kblocks};
    const int pieces = total > 0 ? (static_cast<int>(b1) - 1) / g.kblocks - start.t + 1 : 0;
    // Piece q of this CTA's range (plan.cuh cta_piece, from the range ends above).
    auto piece_of = [&](int q) {
        Piece p;
        p.tile = start.t + q;
        const int t0 = p.tile * g.kblocks;
        p.kb0 = static_cast<int>(b0) > t0 ? static_cast<int>(b0) - t0 : 0;
        p.kb1 = (static_cast<int>(b1) < t0 + g.kblocks ? static_cast<int>(b1) : t0 + g.kblocks) - t0;
        return p;
    };

    // Producer bookkeeping kept for the drain (lane 0 of warp 0).
    uint32_t armed = 0, armed_parity = 0;
    // MMA bookkeeping for the drain (lane 0 of warp 1).
    bool mma_issued = false;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer ----------------
            ptx::prefetch_tensormap(&w_map);
            ptx::prefetch_tensormap(&x_map);
            const uint64_t pol_w = ptx::policy_evict_first();
            const uint64_t pol_x = ptx::policy_evict_last();
            const int npre = total < S ? total : S;
            // Fresh stages: arm them and stream weights before the predecessor ends.
            BlockCursor w = start;
            for (int j = 0; j < npre; ++j) {
                const uint32_t st = sbase + j * L::kStageBytes;
                ptx::mbar_arrive_expect_tx(bar_full + 8 * j, L::kStageBytes);
                armed |= 1u << j;
                ptx::tma_load_2d(st, &w_map, bar_full + 8 * j, w.kb * kBlockK, w.t * kBlockN, pol_w);
                w.next(g.kblocks);
            }
            // The blocks after the ring's worth go to L2 ahead of time.
            const int lead = kShallow ? kL2PrefetchShallow : args.l2_lead;
            const int npf = total - npre < lead ? total - npre : lead;
            BlockCursor pf = w;
            for (int j = 0; j < npf; ++j) {
                ptx::tma_prefetch_l2_2d(&w_map, pf.kb * kBlockK, pf.t * kBlockN);
                pf.next(g.kblocks);
            }
            if (args.l2_after_reduce > 0) {
                // Behind a reduce whose GEMM is complete, HBM would idle until this
                // kernel's wait returns: prefetch more now. Not earlier, where the
                // requests would slow that GEMM's last CTAs.
                const uint64_t t0 = ptx::global_timer_ns();
                bool go = ptx::ld_acquire_gpu(args.gemm_done) != 0u;
                while (!go && ptx::global_timer_ns() - t0 < kAfterReduceWaitNs) {
                    __nanosleep(128);
                    go = ptx::ld_acquire_gpu(args.gemm_done) != 0u;
                }
                if (go) {
                    const int rest = total - npre - npf;
                    const int more = rest < args.l2_after_reduce ? rest : args.l2_after_reduce;
                    for (int j = 0; j < more; ++j) {
                        ptx::tma_prefetch_l2_2d(&w_map, pf.kb * kBlockK, pf.t * kBlockN);
                        pf.next(g.kblocks);
                    }
                }
            }
            if (!LORA) ptx::pdl_wait();  // x may be the predecessor's output
            BlockCursor xc = start;
            for (int j = 0; j < npre; ++j) {
                const uint32_t st = sbase + j * L::kStageBytes;
                ptx::tma_load_2d(st + kWBytes, &x_map, bar_full + 8 * j, xc.kb * kBlockK, 0, pol_x);
                xc.next(g.kblocks);
            }
            int s = npre % S;
            uint32_t ph = npre == S ? 1u : 0u;
            for (int j = npre; j < total; ++j) {
                const int r = bounded_wait(bar_empty + 8 * s, ph ^ 1u, abort_flag, limit);
                if (r != kWaitDone) {
                    if (r == kWaitTimeout) raise_error(args, abort_flag, kErrProducerWait);
                    break;
                }
                const uint32_t st = sbase + s * L::kStageBytes;
                ptx::mbar_arrive_expect_tx(bar_full + 8 * s, L::kStageBytes);
                armed |= 1u << s;
                armed_parity = (armed_parity & ~(1u << s)) | (ph << s);
                ptx::tma_load_2d(st, &w_map, bar_full + 8 * s, w.kb * kBlockK, w.t * kBlockN, pol_w);
                ptx::tma_load_2d(st + kWBytes, &x_map, bar_full + 8 * s, w.kb * kBlockK, 0, pol_x);
                w.next(g.kblocks);
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            constexpr uint32_t idesc = ptx::idesc_bf16_f32(kBlockN, MP);
            if (!LORA) ptx::pdl_wait();  // start the bounded waits' clocks after the predecessor
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            if (args.selftest) {
                // Wait on a barrier nothing ever completes: exercises the bounded wait.
                const int r = bounded_wait(bar_never, 0, abort_flag, limit);
                if (r == kWaitTimeout) raise_error(args, abort_flag, kErrSelftest);
                ok = false;
            }
            for (int q = 0; ok && q < pieces; ++q) {
                const Piece p = piece_of(q);
                const int b = q & 1;
                const uint32_t aph = (q >> 1) & 1;
                int r = bounded_wait(bar_acc_empty + 8 * b, aph ^ 1u, abort_flag, limit);
                if (r != kWaitDone) {
                    if (r == kWaitTimeout) raise_error(args, abort_flag, kErrMmaAccWait);
                    ok = false;
                    break;
                }
                ptx::tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + b * L::kAccCols;
                for (int kb = p.kb0; kb < p.kb1; ++kb) {
                    r = bounded_wait(bar_full + 8 * s, ph, abort_flag, limit);
                    if (r != kWaitDone) {
                        if (r == kWaitTimeout) raise_error(args, abort_flag, kErrMmaFullWait);
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    const uint32_t st = sbase + s * L::kStageBytes;
                    const uint64_t a_desc = ptx::smem_desc_sw128_kmajor(st);
                    const uint64_t b_desc = ptx::smem_desc_sw128_kmajor(st + kWBytes);
#pragma unroll
                    for (int k = 0; k < kBlockK / 16; ++k) {
                        // +32 bytes along K per step: +2 in the address field (>> 4).
                        ptx::mma_bf16(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc,
                                      (kb > p.kb0 || k > 0) ? 1u : 0u);
                    }
                    mma_issued = true;
                    ptx::mma_commit(bar_empty + 8 * s);  // stage free once these MMAs finish
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                ptx::mma_commit(bar_acc_full + 8 * b);
            }
        }
        __syncwarp();
    } else {
        // ---------------- epilogue (128 threads) ----------------
        if (!LORA) ptx::pdl_wait();  // scratch and out may still be in use by the predecessor
        if (args.clear_gemm_done && blockIdx.x == 0 && threadIdx.x == 64) atomicExch(args.gemm_done, 0u);
        const int quarter = warp & 3;              // TMEM lanes 32*quarter .. +31
        const int row = quarter * 32 + lane;       // weight row within the tile
        const int etid = threadIdx.x - 64;
        const int slot_bytes = g.M * kBlockN * static_cast<int>(sizeof(float));
        const int ring_slots = L::kRingBytes / slot_bytes;
        const float *staging = reinterpret_cast<const float *>(smem);
        uint32_t fix_phase = 0;
        bool fix_pending = false;
        // Whole tiles of 32 or 64 padded rows, deep ring, 16-byte aligned output
        // rows: the last piece's tile goes out through the ring.
        constexpr bool kStagedOut = MP >= 32 && !kShallow;
        const bool staged = kStagedOut && (reinterpret_cast<uintptr_t>(args.out) & 15) == 0 &&
                            (g.N & 7) == 0;

        // EPI: the output of this thread's column n of a tile from its FP32 sums, kRows rows at
        // a time (the activations unrolled over all rows would be code that is fetched
        // longer than it runs: 64 rows with a tanh cost 12 us more than without): from
        // tensor memory, or from this thread's column of the idle ring. Rows' residuals are
        // loaded kRows ahead, two to a register, the first before the wait for the accumulator.
        // 4 rows where there may be only one (1 x 2048 x 7168: 9.1 us, 10.0 with 16), 16 where
        // the chains of many overlap (64 x 18432 x 7168, tanh: 44.1 us, 47.8 with 4).
        constexpr int kRows = MP == 16 ? 4 : 16;
        [[maybe_unused]] uint32_t ahead[kRows / 2];
        [[maybe_unused]] float bias = 0.0f;
        auto load_residual = [&](int n, int m0) {
            if (args.epi.residual == nullptr || n >= g.N) return;
            const uint16_t *src = args.epi.residual + static_cast<size_t>(m0) * g.N + n;
#pragma unroll
            for (int i = 0; i < kRows / 2; ++i) {
                const uint32_t lo = m0 + 2 * i < g.M ? src[static_cast<size_t>(2 * i) * g.N] : 0u;
                const uint32_t hi = m0 + 2 * i + 1 < g.M ? src[static_cast<size_t>(2 * i + 1) * g.N] : 0u;
                ahead[i] = lo | (hi << 16);
            }
        };
        // LORA: the rows' adapters and scale A x, the K slices' sums added in order; and the rows
        // of this piece whose part is in tensor memory.
        [[maybe_unused]] int *sm_adapter = reinterpret_cast<int *>(smem + L::kLoraOffset);
        [[maybe_unused]] float *sm_scale = reinterpret_cast<float *>(sm_adapter + kMaxM);
        [[maybe_unused]] float *sm_ax = reinterpret_cast<float *>(smem + L::kLoraAxOffset);
        // How many adapters are in use, and from bit 8 and 16 on which of them (in the order of their
        // first rows) this lane's rows have: one register. 0: shared out by rows.
        [[maybe_unused]] int lora_order = 0;
        [[maybe_unused]] auto lowest = [](uint64_t bits) { return __ffsll(static_cast<long long>(bits)) - 1; };
        // Copied: the adapters in use, each with its rows.
        [[maybe_unused]] uint64_t *sm_rows = reinterpret_cast<uint64_t *>(smem + L::kLoraListOffset);
        [[maybe_unused]] int *sm_used = reinterpret_cast<int *>(smem + L::kLoraListOffset + 8 * kMaxM);
        [[maybe_unused]] const int ring_bytes = (L::kLoraBytes - g.M * args.lora.rank * 4) / 64 * 16;  // of a warp
        [[maybe_unused]] uint8_t *sm_ring = smem + L::kLoraAxOffset + g.M * args.lora.rank * 4 + quarter * ring_bytes;
        [[maybe_unused]] uint64_t lora_rows = 0;
        [[maybe_unused]] const uint32_t lora_taddr =
            tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + L::kLoraCol;
        if constexpr (LORA) {
            const LoraArgs &l = args.lora;
            // The adapters' numbers are as old as x, and the scales are weights: before the wait.
            if (etid < kMaxM) {
                int id = etid < g.M ? __ldcg(l.adapters + etid) : -1;
                if (id >= l.count) id = -1;
                sm_adapter[etid] = id;
                sm_scale[etid] = id >= 0 && l.scales != nullptr ? __ldcg(l.scales + id) : 1.0f;
            }
            ptx::named_barrier_sync(1, kEpilogueThreads);
            // Adapters in the order of their first rows, where the call might go by either form: 0.3 us
            // with 48 rows of rank 32.
            if (kCopied || (MP >= 32 && l.rank >= kLoraCopiedFrom)) {
                constexpr int kHalves = MP > 32 ? 2 : 1;
                int id[kHalves];
                uint64_t rows[kHalves], firsts = 0;  // rows: those with this lane's adapter
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    id[h] = sm_adapter[32 * h + lane];
                    rows[h] = static_cast<uint64_t>(__match_any_sync(0xFFFFFFFFu, id[h])) << 32 * h;
                }
                if constexpr (kHalves == 2) {
                    const int4 *ids = reinterpret_cast<const int4 *>(sm_adapter);
                    auto equal = [](const int4 &at, int to) -> uint32_t {
                        return (at.x == to) | (at.y == to) << 1 | (at.z == to) << 2 | (at.w == to) << 3;
                    };
                    uint32_t upper = 0, lower = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (kCopied) upper |= equal(ids[8 + i], id[0]) << 4 * i;  // direct: only the first is asked for
                        lower |= equal(ids[i], id[1]) << 4 * i;
                    }
                    rows[0] |= static_cast<uint64_t>(upper) << 32;
                    rows[1] |= lower;
                }
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    firsts |= static_cast<uint64_t>(__ballot_sync(0xFFFFFFFFu, id[h] >= 0 && lowest(rows[h]) == 32 * h + lane)) << 32 * h;
                lora_order = __popcll(static_cast<long long>(firsts));
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    const int first = lowest(rows[h]);
                    const int at = __popcll(static_cast<long long>(firsts & ((1ull << first) - 1)));
                    lora_order |= at << (8 + 8 * h);
                    if (kCopied && warp == 2 && id[h] >= 0 && first == 32 * h + lane) {
                        sm_rows[at] = rows[h];
                        sm_used[at] = id[h];
                    }
                }
                if constexpr (kCopied) ptx::named_barrier_sync(1, kEpilogueThreads);
            }
            ptx::pdl_wait();  // A x is the kernel's before
            // Sums of rows without an adapter are not there, and what is read of them is not used.
            const int values = g.M * l.rank;
            auto add_slices = [&](auto at_once, auto slices) {  // loads that are on their way together
                constexpr int kAtOnce = decltype(at_once)::value, kSlices = decltype(slices)::value;
                for (int i0 = etid; i0 < values; i0 += kAtOnce * kEpilogueThreads) {
                    float sum[kAtOnce] = {};
                    for (int s0 = 0; s0 < l.splits; s0 += kSlices) {
                        float v[kSlices][kAtOnce];
#pragma unroll
                        for (int u = 0; u < kSlices; ++u)
#pragma unroll
                            for (int q = 0; q < kAtOnce; ++q) {
                                const int i = i0 + q * kEpilogueThreads;
                                v[u][q] = s0 + u < l.splits && i < values
                                              ? __ldcg(l.sums + static_cast<size_t>(s0 + u) * values + i) : 0.0f;
                            }
#pragma unroll
                        for (int u = 0; u < kSlices; ++u)
#pragma unroll
                            for (int q = 0; q < kAtOnce; ++q) sum[q] = __fadd_rn(sum[q], v[u][q]);
                    }
#pragma unroll
                    for (int q = 0; q < kAtOnce; ++q) {
                        const int i = i0 + q * kEpilogueThreads;
                        if (i < values) sm_ax[i] = __fmul_rn(sum[q], sm_scale[i / l.rank]);
                    }
                }
            };
            if (values <= kEpilogueThreads)
                add_slices(std::integral_constant<int, 1>{}, std::integral_constant<int, 32>{});
            else
                add_slices(std::integral_constant<int, 4>{}, std::integral_constant<int, 8>{});
            ptx::named_barrier_sync(1, kEpilogueThreads);
        }
        // A tile's contributors share its adapters out in turn or, where these are fewer or the call
        // never goes by the other form, its rows of x: the same rows for a contributor in both forms.
        // Direct: the part of column n.
        [[maybe_unused]] auto lora_part = [&](int n, int share, int shares) {
            const LoraArgs &l = args.lora;
            auto wanted = [&](int h) {
                const int m = 32 * h + lane;
                return m < g.M && sm_adapter[m] >= 0 &&
                       ((lora_order & 0xFF) >= shares ? lora_order >> (8 + 8 * h) & 0xFF : m) % shares == share;
            };
            lora_rows = __ballot_sync(0xFFFFFFFFu, wanted(0)) |
                        static_cast<uint64_t>(MP > 32 ? __ballot_sync(0xFFFFFFFFu, wanted(1)) : 0u) << 32;
            constexpr int kAtOnce = MP == 16 ? 4 : 8;  // rows whose loads are on their way together
            const uint16_t *column = l.B + static_cast<size_t>(n < g.N ? n : 0) * l.rank;
            for (uint64_t rest = lora_rows; rest != 0;) {
                uint32_t rows[kAtOnce / 4] = {};  // a byte each
                int count = 0;
                const uint4 *b[kAtOnce];
                float v[kAtOnce][2] = {};
                auto row_of = [&](int u) { return static_cast<int>(rows[u / 4] >> 8 * (u % 4) & 0xFFu); };
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    const int m = rest != 0 ? lowest(rest) : 0;
                    count += rest != 0;
                    rest &= rest - 1;
                    rows[u / 4] |= static_cast<uint32_t>(m) << 8 * (u % 4);
                    const size_t id = u < count ? sm_adapter[m] : 0;
                    b[u] = reinterpret_cast<const uint4 *>(column + id * g.N * l.rank);
                }
                for (int j = 0; j < l.rank; j += 16) {
                    uint4 w[kAtOnce][2];
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            w[u][h] = u < count && j + 8 * h < l.rank ? __ldg(b[u] + j / 8 + h) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        if (u >= count) break;
                        const float4 *ax = reinterpret_cast<const float4 *>(sm_ax + row_of(u) * l.rank + j);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (j + 8 * h >= l.rank) break;
                            const float4 t0 = ax[2 * h], t1 = ax[2 * h + 1];
                            lora_add(v[u], w[u][h], t0, t1);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u)
                    if (u < count) ptx::tmem_st1(lora_taddr + row_of(u), __float_as_uint(__fadd_rn(v[u][0], v[u][1])));
            }
            ptx::tmem_st_wait();
            __syncwarp();
        };
        // Copied: the adapters' part of this thread's column of a tile. A ring entry has the warp's rows of
        // one B, an odd number of 16-byte pieces apart, so that eight rows' pieces lie in different
        // banks. lora_begin: share `share` of `shares`, and the first copies on their way.
        [[maybe_unused]] const int lora_pieces = args.lora.rank / 8;
        [[maybe_unused]] const int lora_pitch = 16 * (lora_pieces + 1 + lora_pieces % 2), lora_entry = 32 * lora_pitch;
        [[maybe_unused]] const int lora_entries = kCopied ? ring_bytes / lora_entry : 0;
        [[maybe_unused]] const int lora_ahead = min(lora_entries - 1, ptx::kMostGroupsAhead);
        [[maybe_unused]] uint64_t lora_mine = 0, lora_copies = 0, lora_uses = 0;  // rows; adapters to copy, to use
        [[maybe_unused]] int lora_put = 0, lora_get = 0, lora_n0 = 0, lora_bound = 0;
        [[maybe_unused]] auto lora_copy = [&]() {
            if (lora_copies != 0) {
                const int a = lowest(lora_copies);
                lora_copies &= lora_copies - 1;
                const uint16_t *from = args.lora.B + (static_cast<size_t>(sm_used[a]) * g.N + lora_n0) * args.lora.rank;
                const unsigned inverse = (65535u + lora_pieces) / lora_pieces;  // p / pieces = p * inverse >> 16, p < 512
                const uint32_t to = ptx::smem_addr(sm_ring) + lora_put * lora_entry;
                for (int p = lane; p < lora_bound; p += 32) {
                    const int r = static_cast<int>(p * inverse >> 16);
                    ptx::cp_async16(to + r * lora_pitch + (p - r * lora_pieces) * 16, from + p * 8);
                }
                lora_put = lora_put + 1 >= lora_entries ? 0 : lora_put + 1;
            }
            ptx::cp_async_commit();  // a group an adapter, empty or not
        };
        [[maybe_unused]] auto lora_begin = [&](int tile, int share, int shares) {
            const int adapters = lora_order & 0xFF;
            lora_mine = ~0ull;
            lora_uses = adapters == 64 ? ~0ull : (1ull << adapters) - 1;
            if (shares > 1) {
                uint64_t every = 0;
                for (int i = share; i < kMaxM; i += shares) every |= 1ull << i;
                if (adapters >= shares) {
                    lora_uses &= every;
                } else {
                    lora_mine = every;
                    for (int a = 0; a < adapters; ++a)
                        if ((sm_rows[a] & every) == 0) lora_uses &= ~(1ull << a);
                }
            }
            lora_copies = lora_uses;
            lora_put = lora_get = 0;
            lora_n0 = tile * kBlockN + quarter * 32;
            lora_bound = (min(lora_n0 + 32, g.N) - lora_n0) * lora_pieces;
            for (int i = 0; i <= lora_ahead; ++i) lora_copy();
        };
        [[maybe_unused]] auto lora_copied = [&]() {
            lora_rows = 0;
            for (; lora_uses != 0; lora_uses &= lora_uses - 1) {
                ptx::cp_async_wait_for(lora_ahead);
                __syncwarp();
                const uint4 *row = reinterpret_cast<const uint4 *>(sm_ring + lora_get * lora_entry + lane * lora_pitch);
                uint64_t rest = sm_rows[lowest(lora_uses)] & lora_mine;
                lora_rows |= rest;
                // Rows of x, `at_once` of them for a pass over the row of B.
                auto rows = [&](auto at_once) {
                    constexpr int kAtOnce = decltype(at_once)::value;
                    const float *ax[kAtOnce];
                    int m[kAtOnce];
                    float v[kAtOnce][2] = {};
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        m[u] = lowest(rest);
                        rest &= rest - 1;
                        ax[u] = sm_ax + m[u] * args.lora.rank;
                    }
#pragma unroll 2
                    for (int c = 0; c < lora_pieces; ++c) {
                        const uint4 w = row[c];
#pragma unroll
                        for (int u = 0; u < kAtOnce; ++u) {
                            const float4 *t = reinterpret_cast<const float4 *>(ax[u]) + 2 * c;
                            lora_add(v[u], w, t[0], t[1]);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) ptx::tmem_st1(lora_taddr + m[u], __float_as_uint(__fadd_rn(v[u][0], v[u][1])));
                };
                int left = __popcll(static_cast<long long>(rest));
                for (; left >= 4; left -= 4) rows(std::integral_constant<int, 4>{});
                if (left & 2) rows(std::integral_constant<int, 2>{});
                if (left & 1) rows(std::integral_constant<int, 1>{});
                lora_get = lora_get + 1 >= lora_entries ? 0 : lora_get + 1;
                __syncwarp();  // the entry is read
                lora_copy();
            }
            ptx::cp_async_wait_for(0);  // nothing but empty groups
            ptx::tmem_st_wait();
            __syncwarp();
        };
        auto emit = [&](int n, bool from_tmem, uint32_t taddr) {
#pragma unroll 1
            for (int m0 = 0; m0 < g.M; m0 += kRows) {
                uint32_t res[kRows / 2], w[kRows];
#pragma unroll
                for (int i = 0; i < kRows / 2; ++i) res[i] = ahead[i];
                if (m0 + kRows < g.M) load_residual(n, m0 + kRows);
                if (from_tmem) {
                    __syncwarp();  // lanes past the right edge went another way; the load is the whole warp's
                    ptx::tmem_ld_now(taddr + m0, w);
                    if constexpr (LORA) {
                        uint32_t part[kRows];
                        ptx::tmem_ld_now(lora_taddr + m0, part);
#pragma unroll
                        for (int i = 0; i < kRows; ++i)
                            if (lora_rows >> (m0 + i) & 1)
                                w[i] = __float_as_uint(__fadd_rn(__uint_as_float(w[i]), __uint_as_float(part[i])));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
                        w[i] = reinterpret_cast<const uint32_t *>(smem)[(m0 + i) * kBlockN + row];
                }
                float v[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    v[i] = __uint_as_float(w[i]);
                    if (args.epi.bias != nullptr) v[i] = __fadd_rn(v[i], bias);
                }
                activate(v, args.epi.activation);
                if (n < g.N) {
                    uint16_t *dst = args.out + static_cast<size_t>(m0) * g.N + n;
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        if (args.epi.residual != nullptr)
                            v[i] = __fadd_rn(v[i], bf16_value((i & 1) ? res[i / 2] >> 16 : res[i / 2] & 0xFFFFu));
                        if (m0 + i < g.M) dst[static_cast<size_t>(i) * g.N] = to_bf16_bits(v[i]);
                    }
                }
            }
            __syncwarp();
        };

        // Finish split tile t. This CTA holds the tile's first K blocks, so the
        // tile is its last piece: its own partial is in registers and the ring
        // is free. Wait until the other contributors have published their
        // partials, pull them into the ring with bulk copies (all in flight at
        // once), add in K (= CTA) order and round once. false = aborted.
        auto finish_tile = [&](int t, int first, int last, const float *own,
                               int first_peer_slot) -> bool {
            float sum[MP];
#pragma unroll
            for (int m = 0; m < MP; ++m) sum[m] = own[m];
            for (int c0 = first + 1; c0 <= last;) {
                const int c1 = last + 1 < c0 + ring_slots ? last + 1 : c0 + ring_slots;
                const int n_in = c1 - c0;
                // The barrier expects every copy of this chunk; one thread per
                // contributor waits for its flag and starts its copy at once, so
                // early partials are on their way while late ones are published.
                if (etid == 0)
                    ptx::mbar_arrive_expect_tx(bar_fix, static_cast<uint32_t>(n_in * slot_bytes));
                fix_pending = true;
                int r = kWaitDone;
                int slot = 0;
                if (etid < n_in) {
                    const int c = c0 + etid;
                    slot = c0 == first + 1 ? first_peer_slot : partial_slot(g, c, t);
                    const unsigned *flag = args.flags + slot;
                    // Acquire loads: the partial behind the flag is visible once it is 1.
                    if (ptx::ld_acquire_gpu(flag) == 0u) {
                        const uint64_t t0 = ptx::global_timer_ns();
                        for (uint32_t spin = 1; ptx::ld_acquire_gpu(flag) == 0u; ++spin) {
                            if ((spin & 15u) == 0) {
                                if (*abort_flag) { r = kWaitAborted; break; }
                                if (ptx::global_timer_ns() - t0 > limit) { r = kWaitTimeout; break; }
                            }
                        }
                    }
                    if (r == kWaitDone) {
                        ptx::fence_proxy_async_global();  // the bulk copy reads what was acquired
                        ptx::bulk_load(sbase + etid * slot_bytes,
                                       args.partials + static_cast<size_t>(slot) * args.slot_floats,
                                       slot_bytes, bar_fix);
                    }
                }
                if (r == kWaitTimeout) raise_error(args, abort_flag, kErrEpilogueWait);
                if (epilogue_any(r != kWaitDone)) return false;
                r = bounded_wait(bar_fix, fix_phase, abort_flag, limit);
                if (r == kWaitTimeout) raise_error(args, abort_flag, kErrEpilogueWait);
                if (epilogue_any(r != kWaitDone)) return false;
                fix_pending = false;
                fix_phase ^= 1u;
                for (int c = c0; c < c1; ++c) {
                    const float *src = staging + static_cast<size_t>(c - c0) * g.M * kBlockN + row;
#pragma unroll
                    for (int m = 0; m < MP; ++m)
                        if (m < g.M) sum[m] = __fadd_rn(sum[m], src[m * kBlockN]);
                }
                // The partials are consumed: re-arm their flags for the next call.
                if (etid < n_in) args.flags[slot] = 0u;
                ptx::named_barrier_sync(1, kEpilogueThreads);  // the ring is refilled next
                c0 = c1;
            }
            const int n = t * kBlockN + row;
            if constexpr (EPI) {
#pragma unroll
                for (int m = 0; m < MP; ++m)
                    if (m < g.M) reinterpret_cast<float *>(smem)[m * kBlockN + row] = sum[m];
                emit(n, false, 0u);
                return true;
            }
            if (n < g.N) {
#pragma unroll
                for (int m = 0; m < MP; ++m)
                    if (m < g.M)
                        args.out[static_cast<size_t>(m) * g.N + n] = to_bf16_bits(output_value(sum[m], args));
            }
            return true;
        };

        for (int q = 0; q < pieces; ++q) {
            const Piece p = piece_of(q);
            // The plan's arithmetic (64-bit divisions) before the wait, not on
            // the split-K tail after it.
            int first, last;
            tile_contributors(g, p.tile, first, last);
            const int my_slot = 2 * cta + (p.tile == start.t ? 0 : 1);  // plan.cuh partial_slot
            const int first_peer_slot =
                first + 1 + etid <= last ? partial_slot(g, first + 1 + etid, p.tile) : 0;
            // A piece from the tile's first K block on is the one that stores the tile.
            if (EPI && p.kb0 == 0 && !args.publish_only) {
                const int n = p.tile * kBlockN + row;
                if (args.epi.bias != nullptr && n < g.N) bias = bf16_value(args.epi.bias[n]);
                load_residual(n, 0);
            }
            if constexpr (kCopied) {
                lora_begin(p.tile, cta - first, last - first + 1);
                lora_copied();
            } else if constexpr (LORA != kNoLora) {
                lora_part(p.tile * kBlockN + row, cta - first, last - first + 1);
            }
            const int b = q & 1;
            const uint32_t aph = (q >> 1) & 1;
            const int r = bounded_wait(bar_acc_full + 8 * b, aph, abort_flag, limit);
            if (r == kWaitTimeout) raise_error(args, abort_flag, kErrEpilogueWait);
            if (epilogue_any(r != kWaitDone)) break;
            ptx::tc_fence_after_sync();
            if constexpr (EPI) {
                if (p.kb0 == 0 && p.kb1 == g.kblocks && !args.publish_only) {
                    emit(p.tile * kBlockN + row, true,
                         tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + b * L::kAccCols);
                    ptx::tc_fence_before_sync();
                    ptx::mbar_arrive(bar_acc_empty + 8 * b);  // the MMA may reuse this buffer
                    continue;
                }
            }
            float acc[MP];
            {
                const uint32_t taddr =
                    tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + b * L::kAccCols;
#pragma unroll
                for (int c = 0; c < MP; c += 16) {
                    uint32_t v[16];
                    ptx::tmem_ld16(taddr + c, v);
                    ptx::tmem_ld_wait(v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c + i] = __uint_as_float(v[i]);
                    if constexpr (LORA) {
                        ptx::tmem_ld_now(lora_taddr + c, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (lora_rows >> (c + i) & 1) acc[c + i] = __fadd_rn(acc[c + i], __uint_as_float(v[i]));
                    }
                }
            }
            ptx::tc_fence_before_sync();
            ptx::mbar_arrive(bar_acc_empty + 8 * b);  // the MMA may reuse this buffer

            const int n = p.tile * kBlockN + row;
            if (p.kb0 == 0 && p.kb1 == g.kblocks && !args.publish_only) {
                // Whole tile in this CTA: round once and store.
                if (kStagedOut && staged && q == pieces - 1) {
#pragma unroll
                    for (int m = 0; m < MP; ++m) acc[m] = output_value(acc[m], args);
                    store_tile_staged<MP>(acc, args.out, g.M, g.N, p.tile, row, etid, sbase);
                    continue;
                }
                if (n < g.N) {
#pragma unroll
                    for (int m = 0; m < MP; ++m)
                        if (m < g.M)
                            args.out[static_cast<size_t>(m) * g.N + n] =
                                to_bf16_bits(output_value(acc[m], args));
                }
                continue;
            }
            if (first == cta && !args.publish_only) {
                // The tile starts in this CTA's range: this CTA finishes it.
                if (!finish_tile(p.tile, first, last, acc, first_peer_slot)) break;
                continue;
            }
            // Publish this CTA's partial: the values, then a release flag. The
            // finishing CTA reads them with bulk copies (the async proxy).
            float *mine = args.partials + static_cast<size_t>(my_slot) * args.slot_floats;
#pragma unroll
            for (int m = 0; m < MP; ++m)
                if (m < g.M) __stcg(mine + m * kBlockN + row, acc[m]);
            if (args.publish_only) continue;  // read by the next kernel, after this grid
            ptx::fence_proxy_async_global();
            ptx::named_barrier_sync(1, kEpilogueThreads);
            // One release store after the barrier covers every thread's stores of
            // the partial (the barrier orders them before it).
            if (etid == 0) {
                ptx::st_release_gpu(args.flags + my_slot, 1u);
            }
        }
        if (fix_pending) {
            // Copies still in flight must land before the CTA's memory is released.
            const uint64_t t0 = ptx::global_timer_ns();
            while (!ptx::mbar_try_wait(bar_fix, fix_phase)) {
                if (ptx::global_timer_ns() - t0 > kDrainLimitNs) {
                    record_error(args, kErrDrain);
                    break;
                }
            }
        }
    }

    // ---------------- teardown ----------------
    __syncthreads();
    if (*abort_flag) {
        // Nothing may still write this CTA's shared or tensor memory when it exits.
        if (warp == 0 && lane == 0) {
            for (int s = 0; s < S; ++s) {
                if (!(armed & (1u << s))) continue;
                const uint32_t par = (armed_parity >> s) & 1u;
                const uint64_t t0 = ptx::global_timer_ns();
                while (!ptx::mbar_try_wait(bar_full + 8 * s, par)) {
                    if (ptx::global_timer_ns() - t0 > kDrainLimitNs) {
                        record_error(args, kErrDrain);
                        break;
                    }
                }
            }
        }
        if (warp == 1 && lane == 0 && mma_issued) {
            ptx::mma_commit(bar_drain);
            const uint64_t t0 = ptx::global_timer_ns();
            while (!ptx::mbar_try_wait(bar_drain, 0)) {
                if (ptx::global_timer_ns() - t0 > kDrainLimitNs) {
                    record_error(args, kErrDrain);
                    break;
                }
            }
        }
        __syncthreads();
    }
    if (warp == 0) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem_base, L::kTmemCols);
    }
}

template <int MP, int STAGES, bool EPI, int LORA>
cudaError_t launch_kernel(const CUtensorMap &w_map, const CUtensorMap &x_map,
                           const GemmArgs &args, int ctas, cudaStream_t stream, bool pdl,
                           int device) {
    using L = Layout<MP, STAGES, LORA>;
    constexpr int kMostBytes = L::kDynamicBytes + (LORA == kLoraDirect ? MP * kLoraMaxRank * 4 : 0);
    static_assert(kMostBytes <= 232448, "shared memory of a CTA");
    static bool configured[64] = {};
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    if (!configured[device]) {
        cudaError_t e = cudaFuncSetAttribute(decode_gemm_kernel<MP, STAGES, EPI, LORA>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMostBytes);
        if (e != cudaSuccess) return e;
        configured[device] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = L::kDynamicBytes + (LORA == kLoraDirect ? args.M * args.lora.rank * 4 : 0);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // LORA: always, behind the library's own first half (whatever comes before that is
    // waited for there).
    cfg.numAttrs = pdl || LORA ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, decode_gemm_kernel<MP, STAGES, EPI, LORA>, w_map, x_map, args);
}

template <int MP, int STAGES>
cudaError_t launch_variant(const CUtensorMap &w_map, const CUtensorMap &x_map,
                           const GemmArgs &args, int ctas, cudaStream_t stream, bool pdl,
                           int device) {
    if (args.lora.rank > 0) {
        if constexpr (MP >= 32 && STAGES > kMaxShallowStages)
            if (args.lora.rank >= 64 || (args.lora.rank >= kLoraCopiedFrom && args.lora.rank * args.M >= 96 * args.lora.count))
                return launch_kernel<MP, MP == 64 ? 6 : 8, true, kLoraCopied>(w_map, x_map, args, ctas, stream, pdl, device);
        // A x takes one stage of the rings that fill the shared memory (up to 32 KB).
        constexpr int kLoraStages = STAGES - (MP >= 32 && STAGES > kMaxShallowStages ? 1 : 0);
        return launch_kernel<MP, kLoraStages, true, kLoraDirect>(w_map, x_map, args, ctas, stream, pdl, device);
    }
    if (args.epilogue)
        return launch_kernel<MP, STAGES, true, kNoLora>(w_map, x_map, args, ctas, stream, pdl, device);
    return launch_kernel<MP, STAGES, false, kNoLora>(w_map, x_map, args, ctas, stream, pdl, device);
}

// Deep rings: about 185 KB for 16 rows, near the 227 KB a CTA may use for 32 and
// 64 rows (their x slices take a larger share of each stage). Measured on GB300:
// 12 stages for 16 rows gain alone but lose inside the layer chain.
constexpr int kDeepStages16 = 10, kDeepStages32 = 11, kDeepStages64 = 9;
// Shallow rings sized so two CTAs fit on one SM (about 112 and 104 KB). Rows of
// x above 32 always take the deep ring (plan.cuh): a 4-stage shallow ring for
// them measured 0.6-1 us slower on GB300 even on short streams.
constexpr int kShallowStages16 = 6, kShallowStages32 = 5;
static_assert(kShallowStages16 <= kMaxShallowStages && kDeepStages64 > kMaxShallowStages,
              "ring classes must stay apart");

}  // namespace

int gemm_stages(int mma_n, bool shallow) {
    if (mma_n == 64) return kDeepStages64;
    if (shallow) return mma_n == 16 ? kShallowStages16 : kShallowStages32;
    return mma_n == 16 ? kDeepStages16 : kDeepStages32;
}

int gemm_smem_bytes(int mma_n, bool shallow) {
    if (mma_n == 16)
        return shallow ? Layout<16, kShallowStages16>::kDynamicBytes : Layout<16, kDeepStages16>::kDynamicBytes;
    if (mma_n == 32)
        return shallow ? Layout<32, kShallowStages32>::kDynamicBytes : Layout<32, kDeepStages32>::kDynamicBytes;
    return Layout<64, kDeepStages64>::kDynamicBytes;
}

cudaError_t launch_decode_gemm(const CUtensorMap &w_map, const CUtensorMap &x_map,
                               const GemmArgs &args, int mma_n, int ctas, cudaStream_t stream,
                               bool pdl, bool shallow, int device) {
    if (mma_n == 16) {
        if (shallow) return launch_variant<16, kShallowStages16>(w_map, x_map, args, ctas, stream, pdl, device);
        return launch_variant<16, kDeepStages16>(w_map, x_map, args, ctas, stream, pdl, device);
    }
    if (mma_n == 32) {
        if (shallow) return launch_variant<32, kShallowStages32>(w_map, x_map, args, ctas, stream, pdl, device);
        return launch_variant<32, kDeepStages32>(w_map, x_map, args, ctas, stream, pdl, device);
    }
    return launch_variant<64, kDeepStages64>(w_map, x_map, args, ctas, stream, pdl, device);
}

}  // namespace skinny

// ---- scratch in a static device array (for decode_gemm_bf16_noalloc) -----------------
//
// The same kernel can run with its split-K scratch in this file-scope array
// instead of memory from cudaMalloc. Sized for kStaticScratchCtas CTAs with
// partial tiles of up to 32 rows: 2 slots per CTA, then one flag per slot, then
// the error word. Every GPU that loads the library holds it until the process
// exits.
namespace skinny {
namespace {

constexpr size_t kStaticPartialBytes =
    static_cast<size_t>(2) * kStaticScratchCtas * kStaticSlotRows * kBlockN * sizeof(float);
constexpr size_t kStaticFlagBytes = 2048;  // >= 2 * kStaticScratchCtas flags, 256-aligned
constexpr size_t kStaticScratchBytes = kStaticPartialBytes + kStaticFlagBytes + 256;
static_assert(2 * kStaticScratchCtas * sizeof(unsigned) <= kStaticFlagBytes, "flag space");

static __device__ __align__(256) unsigned char g_static_scratch[kStaticScratchBytes];

std::mutex g_static_mutex;
void *g_static_base[64] = {};

}  // namespace

cudaError_t static_scratch_for_current_device(StaticScratch *out) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_static_mutex);
    if (g_static_base[dev] == nullptr) {
        // Host code sees g_static_scratch only as a stand-in symbol; the array's
        // device address has to be looked up, once per device, with it current.
        void *p = nullptr;
        e = cudaGetSymbolAddress(&p, g_static_scratch);
        if (e != cudaSuccess) return e;
        if (p == nullptr) return cudaErrorInvalidSymbol;
        g_static_base[dev] = p;
    }
    char *base = static_cast<char *>(g_static_base[dev]);
    out->partials = reinterpret_cast<float *>(base);
    out->flags = reinterpret_cast<unsigned *>(base + kStaticPartialBytes);
    out->err = reinterpret_cast<int *>(base + kStaticPartialBytes + kStaticFlagBytes);
    out->zero_bytes = kStaticFlagBytes + sizeof(int);  // flags and error word
    out->max_ctas = kStaticScratchCtas;
    return cudaSuccess;
}

}  // namespace skinny
