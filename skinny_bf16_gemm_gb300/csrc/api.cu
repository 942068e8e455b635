// The library's C ABI (include/skinny.h): argument checks, the per-device state
// (SM count, split-K scratch, error word), TMA descriptor encoding and launches.
// Every check runs before any launch; a rejected call touches nothing.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "attention_plan.cuh"
#include "kernels.h"
#include "plan.cuh"
#include "skinny.h"

namespace skinny {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxHeads = 1024;
constexpr int kMaxHeadDim = 256;
constexpr unsigned long long kWaitLimitNs = 1000000000ull;  // 1 s per internal wait

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
    // A host-mapped word the decode GEMM sets when one of its waits runs out:
    // the host reads it without synchronising, so the next call can refuse to
    // run on scratch a kernel left half used (host_err) -- and the kernel's
    // address of it (host_err_dev).
    int *host_err = nullptr;
    int *host_err_dev = nullptr;
};

std::mutex g_mutex;
DeviceState g_devices[kMaxDevices];
bool g_pdl = false;  // programmatic dependent launch, opt-in (skinny_set_pdl)
int g_l2_lead = kL2LeadDefault;  // decode GEMM deep-ring L2 lead (skinny_set_l2_prefetch)

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

int current_device(int *dev) {
    if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) {
        cudaGetLastError();
        return SKINNY_ERR_DEVICE;
    }
    return SKINNY_OK;
}

// Device properties (once per device). Caller holds g_mutex.
int device_state_locked(int dev, DeviceState **out) {
    DeviceState &d = g_devices[dev];
    if (!d.ready) {
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
            cudaGetLastError();
            return SKINNY_ERR_DEVICE;
        }
        d.ready = true;
    }
    // The kernels are built for sm_103a only.
    if (d.major != 10 || d.minor != 3) return SKINNY_ERR_DEVICE;
    *out = &d;
    return SKINNY_OK;
}

int device_state(int dev, DeviceState **out) {
    std::lock_guard<std::mutex> lock(g_mutex);
    return device_state_locked(dev, out);
}

// The decode GEMM's scratch: allocated and zeroed once per device.
int ensure_scratch(int dev, cudaStream_t stream, DeviceState **out) {
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceState *d = nullptr;
    int st = device_state_locked(dev, &d);
    if (st != SKINNY_OK) return st;
    if (d->scratch == nullptr) {
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) {
            cudaGetLastError();
            return SKINNY_ERR_LAUNCH;
        }
        if (cap != cudaStreamCaptureStatusNone) return SKINNY_ERR_CAPTURE;
        const size_t partial_bytes = static_cast<size_t>(2) * d->sms * kSlotFloats * sizeof(float);
        const size_t flag_bytes = (static_cast<size_t>(2) * d->sms * sizeof(unsigned) + 255) / 256 * 256;
        const size_t bytes = partial_bytes + flag_bytes + 256;
        void *p = nullptr;
        if (cudaMalloc(&p, bytes) != cudaSuccess) {
            cudaGetLastError();
            return SKINNY_ERR_ALLOC;
        }
        if (cudaMemset(p, 0, bytes) != cudaSuccess) {
            cudaGetLastError();
            cudaFree(p);
            return SKINNY_ERR_ALLOC;
        }
        void *h = nullptr, *hd = nullptr;
        if (cudaHostAlloc(&h, 256, cudaHostAllocMapped | cudaHostAllocPortable) != cudaSuccess) {
            cudaGetLastError();
            cudaFree(p);
            return SKINNY_ERR_ALLOC;
        }
        if (cudaHostGetDevicePointer(&hd, h, 0) != cudaSuccess) {
            cudaGetLastError();
            cudaFreeHost(h);
            cudaFree(p);
            return SKINNY_ERR_ALLOC;
        }
        std::memset(h, 0, 256);
        d->host_err = static_cast<int *>(h);
        d->host_err_dev = static_cast<int *>(hd);
        d->scratch = p;
        d->partials = static_cast<float *>(p);
        d->flags = reinterpret_cast<unsigned *>(static_cast<char *>(p) + partial_bytes);
        d->err = reinterpret_cast<int *>(static_cast<char *>(p) + partial_bytes + flag_bytes);
        d->flag_bytes = flag_bytes;
        d->gemm_done = reinterpret_cast<unsigned *>(d->err) + 32;
    }
    *out = d;
    return SKINNY_OK;
}

int encoder(EncodeTiledFn *fn) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_encode == nullptr) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || p == nullptr) {
            cudaGetLastError();
            return SKINNY_ERR_DEVICE;
        }
        g_encode = reinterpret_cast<EncodeTiledFn>(p);
    }
    *fn = g_encode;
    return SKINNY_OK;
}

// The pointer must be device (or managed) memory of device `dev`.
int check_device_pointer(const void *p, int dev) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_DEVICE;
    }
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) return SKINNY_ERR_DEVICE;
    if (a.device != dev) return SKINNY_ERR_DEVICE;
    return SKINNY_OK;
}

bool overlaps(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bn && b0 < a0 + an;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// 2-D BF16 tensor map over a row-major [rows, cols] array, box [box_rows, 64].
int encode_2d(EncodeTiledFn enc, CUtensorMap *map, const void *base, uint64_t rows,
              uint64_t cols, uint32_t box_rows) {
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * 2};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBlockK), box_rows};
    const cuuint32_t estride[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims,
                     strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SKINNY_OK : SKINNY_ERR_LAUNCH;
}

int gemm_shape_ok(int M, int N, int K) {
    if (M < 1 || M > kMaxM || N < 1 || K < 8 || (K % 8) != 0) return SKINNY_ERR_SHAPE;
    // The kernel counts 128 x 64 weight blocks in 32-bit integers (a weight of
    // 2^31 blocks would be 32 TiB).
    const long long blocks = static_cast<long long>((N + kBlockN - 1) / kBlockN) *
                             ((K + kBlockK - 1) / kBlockK);
    if (blocks >= (1ll << 31)) return SKINNY_ERR_SHAPE;
    return SKINNY_OK;
}

int mma_n_for(int M) { return M <= 16 ? 16 : (M <= 32 ? 32 : 64); }

// SKINNY_ERR_TIMEOUT while a decode GEMM on this device has recorded a wait that
// ran out and skinny_device_error() has not cleared it: the split-K scratch
// may hold flags that kernel never consumed, so nothing that uses it runs.
int pending_timeout(const DeviceState *d) {
    if (d->host_err != nullptr && *reinterpret_cast<volatile const int *>(d->host_err) != 0)
        return SKINNY_ERR_TIMEOUT;
    return SKINNY_OK;
}

// The launch settings of one call: the caller's options where given, else the
// process-wide settings (skinny_set_pdl, skinny_set_l2_prefetch).
struct LaunchSettings {
    bool pdl;
    int l2_lead;
    int l2_after_reduce;
};

int resolve_settings(const skinny_launch_opts *opts, LaunchSettings *out) {
    if (opts != nullptr) {
        if (opts->pdl < SKINNY_OPT_DEFAULT || opts->pdl > 1) return SKINNY_ERR_ARG;
        if (opts->l2_prefetch < SKINNY_OPT_DEFAULT || opts->l2_prefetch > kL2LeadMax)
            return SKINNY_ERR_ARG;
        if (opts->l2_after_reduce < SKINNY_OPT_DEFAULT || opts->l2_after_reduce > kL2LeadMax)
            return SKINNY_ERR_ARG;
    }
    std::lock_guard<std::mutex> lock(g_mutex);
    out->pdl = g_pdl;
    out->l2_lead = g_l2_lead;
    out->l2_after_reduce = 0;
    if (opts != nullptr) {
        if (opts->pdl != SKINNY_OPT_DEFAULT) out->pdl = opts->pdl != 0;
        if (opts->l2_prefetch != SKINNY_OPT_DEFAULT) out->l2_lead = opts->l2_prefetch;
        if (opts->l2_after_reduce > 0) out->l2_after_reduce = opts->l2_after_reduce;
    }
    return SKINNY_OK;
}

int gemm_launch(const void *x, const void *W, void *out, int M, int N, int K, void *stream,
                const skinny_launch_opts *opts, int selftest, unsigned long long limit_ns,
                int logits = 0, float soft_cap = 0.0f, float scale = 1.0f,
                const Epilogue *epi = nullptr) {
    if (!x || !W || !out) return SKINNY_ERR_NULL;
    int st = gemm_shape_ok(M, N, K);
    if (st) return st;
    const void *bias = epi ? epi->bias : nullptr, *residual = epi ? epi->residual : nullptr;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(out, 2) || !aligned(bias, 2) ||
        !aligned(residual, 2))
        return SKINNY_ERR_ALIGN;
    const size_t xb = static_cast<size_t>(M) * K * 2, wb = static_cast<size_t>(N) * K * 2,
                 ob = static_cast<size_t>(M) * N * 2;
    // out may be the residual itself (element-wise in place), nothing else.
    if (overlaps(out, ob, x, xb) || overlaps(out, ob, W, wb) ||
        (bias && overlaps(out, ob, bias, static_cast<size_t>(N) * 2)) ||
        (residual && residual != out && overlaps(out, ob, residual, ob)))
        return SKINNY_ERR_ALIAS;
    LaunchSettings ls;
    if ((st = resolve_settings(opts, &ls))) return st;
    int dev;
    if ((st = current_device(&dev))) return st;
    if ((st = check_device_pointer(x, dev)) || (st = check_device_pointer(W, dev)) ||
        (st = check_device_pointer(out, dev)) ||
        (bias && (st = check_device_pointer(bias, dev))) ||
        (residual && residual != out && (st = check_device_pointer(residual, dev))))
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceState *d = nullptr;
    if ((st = ensure_scratch(dev, s, &d))) return st;
    if ((st = pending_timeout(d))) return st;
    EncodeTiledFn enc;
    if ((st = encoder(&enc))) return st;
    const int mma_n = mma_n_for(M);
    alignas(64) CUtensorMap w_map, x_map;
    if ((st = encode_2d(enc, &w_map, W, N, K, kBlockN))) return st;
    if ((st = encode_2d(enc, &x_map, x, M, K, mma_n))) return st;
    const GemmGeometry g = make_geometry(M, N, K, choose_ctas(N, d->sms));
    GemmArgs a = {};
    a.M = M;
    a.N = N;
    a.K = K;
    a.out = static_cast<uint16_t *>(out);
    a.partials = d->partials;
    a.slot_floats = kSlotFloats;
    a.flags = d->flags;
    a.err = d->err;
    a.host_err = d->host_err_dev;
    a.wait_limit_ns = limit_ns;
    a.selftest = selftest;
    a.logits = logits;
    a.soft_cap = soft_cap;
    a.scale = scale;
    if (epi) {
        a.epilogue = 1;
        a.epi = *epi;
    }
    const bool pdl = ls.pdl;
    a.l2_lead = ls.l2_lead;
    a.gemm_done = d->gemm_done;
    a.l2_after_reduce = ls.l2_after_reduce;
    // Split tiles of 64-row accumulators, every CTA within at most two tiles (two
    // scratch slots), plain output: the GEMM only publishes its partials and a
    // small kernel finishes them (same order, same bits). A finisher CTA would
    // pull 32 KB partial slots through its ring and add 64 rows per thread; the
    // finish kernel spreads that over every column. Measured on GB300: 2 µs
    // faster at M = 64, N = 7168, K = 14336; slower for 16 and 32 rows, where the
    // extra kernel boundary costs more than the in-kernel finish.
    int split = 0;
    for (int t = 0; t < g.tiles && !split; ++t) {
        int first, last;
        tile_contributors(g, t, first, last);
        split = first != last;
    }
    if (split && mma_n == 64 && g.ctas >= g.tiles && !logits && !selftest) {
        a.publish_only = 1;
        cudaError_t e = launch_decode_gemm(w_map, x_map, a, mma_n, g.ctas, s, pdl,
                                           use_shallow_ring(g, pdl), dev);
        if (e == cudaSuccess) {
            SplitKPartials fix = {};
            fix.partials = d->partials;
            fix.slot_floats = kSlotFloats;
            fix.M = M;
            fix.N = N;
            fix.K = K;
            fix.ctas = g.ctas;
            e = launch_splitk_finish(fix, static_cast<uint16_t *>(out), epi, s, pdl);
        }
        if (e != cudaSuccess) {
            cudaGetLastError();
            return SKINNY_ERR_LAUNCH;
        }
        return SKINNY_OK;
    }
    cudaError_t e = launch_decode_gemm(w_map, x_map, a, mma_n, g.ctas, s, pdl,
                                       use_shallow_ring(g, pdl), dev);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

// decode_gemm_bf16 with its split-K scratch in the static device array of
// decode_gemm.cu: no device memory is allocated on this path.
int gemm_launch_static(const void *x, const void *W, void *out, int M, int N, int K,
                       void *stream) {
    if (!x || !W || !out) return SKINNY_ERR_NULL;
    int st = gemm_shape_ok(M, N, K);
    if (st) return st;
    if (M > kStaticSlotRows) return SKINNY_ERR_SHAPE;  // the static partial tiles hold 32 rows
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(out, 2)) return SKINNY_ERR_ALIGN;
    const size_t xb = static_cast<size_t>(M) * K * 2, wb = static_cast<size_t>(N) * K * 2,
                 ob = static_cast<size_t>(M) * N * 2;
    if (overlaps(out, ob, x, xb) || overlaps(out, ob, W, wb)) return SKINNY_ERR_ALIAS;
    int dev;
    if ((st = current_device(&dev))) return st;
    DeviceState *d = nullptr;
    if ((st = device_state(dev, &d))) return st;
    if ((st = check_device_pointer(x, dev)) || (st = check_device_pointer(W, dev)) ||
        (st = check_device_pointer(out, dev)))
        return st;
    StaticScratch sc;
    if (static_scratch_for_current_device(&sc) != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_DEVICE;
    }
    EncodeTiledFn enc;
    if ((st = encoder(&enc))) return st;
    const int mma_n = mma_n_for(M);
    alignas(64) CUtensorMap w_map, x_map;
    if ((st = encode_2d(enc, &w_map, W, N, K, kBlockN))) return st;
    if ((st = encode_2d(enc, &x_map, x, M, K, mma_n))) return st;
    // At most as many CTAs as the array has partial-tile slots for.
    const int ctas = choose_ctas(N, d->sms);
    const GemmGeometry g = make_geometry(M, N, K, ctas < sc.max_ctas ? ctas : sc.max_ctas);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // The array keeps the previous call's contents: the published-partial flags
    // and the error word must start this call at zero.
    if (cudaMemsetAsync(sc.flags, 0, sc.zero_bytes, s) != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    GemmArgs a = {};
    a.M = M;
    a.N = N;
    a.K = K;
    a.out = static_cast<uint16_t *>(out);
    a.partials = sc.partials;
    a.slot_floats = kStaticSlotRows * kBlockN;
    a.flags = sc.flags;
    a.err = sc.err;
    a.wait_limit_ns = kWaitLimitNs;
    a.selftest = 0;
    a.logits = 0;
    a.soft_cap = 0.0f;
    a.scale = 1.0f;
    bool pdl;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        pdl = g_pdl;
        a.l2_lead = g_l2_lead;
    }
    cudaError_t e = launch_decode_gemm(w_map, x_map, a, mma_n, g.ctas, s, pdl,
                                       use_shallow_ring(g, pdl), dev);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

// CTAs per row of the reduce. An 8-CTA cluster per row spreads a few rows, or
// heavy ones, over many SMs; with enough light rows one 896-thread CTA per row is
// faster (no cluster exchange). Loads per thread = TP partial fragments plus the
// residual's. Chosen from a sweep of 1, 2, 4 and 8 CTAs per row over TP in
// {2, 4, 8}, M in {1, .., 64}, residual or not, on GB300.
int reduce_ctas_per_row(int M, int TP, bool residual) {
    const int loads = TP + (residual ? 1 : 0);
    if ((M >= 32 && loads <= 8) || (M >= 16 && loads <= 4)) return 1;
    return 8;
}

// The reduce's argument checks that need no device: pointers, shapes, eps,
// alignment, aliasing.
int reduce_arg_checks(const void *partials, int TP, const void *residual, const void *gamma,
                      const void *out, const void *residual_out, int M, float eps) {
    if (!partials || !gamma || !out || !residual_out) return SKINNY_ERR_NULL;
    if (TP < 1 || TP > SKINNY_REDUCE_MAX_TP || M < 1 || M > SKINNY_REDUCE_MAX_M)
        return SKINNY_ERR_SHAPE;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return SKINNY_ERR_ARG;
    if (!aligned(partials, 16) || !aligned(gamma, 16) || !aligned(out, 16) ||
        !aligned(residual_out, 16) || (residual && !aligned(residual, 16)))
        return SKINNY_ERR_ALIGN;
    const size_t row = static_cast<size_t>(M) * SKINNY_HIDDEN * 2;
    const size_t pb = row * TP, gb = SKINNY_HIDDEN * 2;
    if (overlaps(out, row, residual_out, row) || overlaps(out, row, partials, pb) ||
        overlaps(out, row, gamma, gb) || overlaps(residual_out, row, partials, pb) ||
        overlaps(residual_out, row, gamma, gb) || (residual && overlaps(out, row, residual, row)))
        return SKINNY_ERR_ALIAS;
    // residual_out may be residual itself (element-wise in-place), nothing else.
    if (residual && residual != residual_out && overlaps(residual_out, row, residual, row))
        return SKINNY_ERR_ALIAS;
    return SKINNY_OK;
}

// The current device, and the reduce's pointers on it.
int reduce_device_checks(const void *partials, const void *residual, const void *gamma,
                         const void *out, const void *residual_out, int *dev) {
    int st;
    if ((st = current_device(dev))) return st;
    DeviceState *d = nullptr;
    if ((st = device_state(*dev, &d))) return st;
    if ((st = check_device_pointer(partials, *dev)) || (st = check_device_pointer(gamma, *dev)) ||
        (st = check_device_pointer(out, *dev)) || (st = check_device_pointer(residual_out, *dev)) ||
        (residual && (st = check_device_pointer(residual, *dev))))
        return st;
    return SKINNY_OK;
}

int log2_or_minus_one(int n) { return (n & (n - 1)) == 0 ? __builtin_ctz(n) : -1; }

// Bytes from a row's first element to past the last row's last.
size_t row_span(int rows, long long stride, long long width) {
    return (static_cast<size_t>(rows - 1) * stride + width) * 2;
}

// Whether a pool that is written has two elements in one place. Its axes must lie within each
// other: each stride clears all that the smaller ones reach. The values then meet the keys
// where their distance is a sum of steps along the axes, give or take a head: at each axis,
// the largest first, only the two numbers of steps around the distance can come near enough.
struct PoolAxis {
    long long stride;
    int size;
};
bool steps_meet(long long distance, const PoolAxis *axes, int n, int head_dim) {
    if (n == 0) return distance > -head_dim && distance < head_dim;
    const long long s = axes[n - 1].stride;
    const long long below = distance >= 0 ? distance / s : -((-distance + s - 1) / s);
    for (long long t = below; t <= below + 1; ++t)
        if (t > -axes[n - 1].size && t < axes[n - 1].size && steps_meet(distance - t * s, axes, n - 1, head_dim))
            return true;
    return false;
}
bool pool_meets_itself(const skinny_kv_cache *c) {
    PoolAxis axes[3];
    int n = 0;
    for (const PoolAxis &a : {PoolAxis{c->page_stride, c->num_pages}, PoolAxis{c->token_stride, c->page_size},
                              PoolAxis{c->head_stride, c->kv_heads}})
        if (a.size > 1) axes[n++] = a;
    std::sort(axes, axes + n, [](const PoolAxis &a, const PoolAxis &b) { return a.stride < b.stride; });
    long long extent = c->head_dim;
    for (int i = 0; i < n; ++i) {
        if (axes[i].stride < extent) return true;
        extent += axes[i].stride * (axes[i].size - 1);
    }
    const uintptr_t k = reinterpret_cast<uintptr_t>(c->k), v = reinterpret_cast<uintptr_t>(c->v);
    const unsigned long long apart = (k < v ? v - k : k - v) / 2;
    return apart < static_cast<unsigned long long>(extent) &&
           steps_meet(static_cast<long long>(apart), axes, n, c->head_dim);
}

// A cache's own rules, and the bytes its keys (or values) span.
int check_cache(const skinny_kv_cache *c, bool write, size_t *span) {
    if (!c->k || !c->v) return SKINNY_ERR_NULL;
    if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->kv_heads > kMaxHeads ||
        c->head_dim < 8 || c->head_dim > kMaxHeadDim || c->head_dim % 8 != 0)
        return SKINNY_ERR_SHAPE;
    const long long strides[3] = {c->page_stride, c->token_stride, c->head_stride};
    const int sizes[3] = {c->num_pages, c->page_size, c->kv_heads};
    unsigned long long last = 0;
    for (int i = 0; i < 3; ++i) {
        if (strides[i] < 0 || strides[i] > (1ll << 40)) return SKINNY_ERR_SHAPE;
        if (strides[i] % 8 != 0) return SKINNY_ERR_ALIGN;
        // At most 3 * 2^31 * 2^40: no overflow of the unsigned 128-bit sum.
        const unsigned __int128 more = static_cast<unsigned __int128>(sizes[i] - 1) * strides[i];
        if (more > (1ull << 44)) return SKINNY_ERR_SHAPE;
        last += static_cast<unsigned long long>(more);
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SKINNY_ERR_ALIGN;
    if (write && pool_meets_itself(c)) return SKINNY_ERR_ALIAS;
    *span = static_cast<size_t>(last + c->head_dim) * 2;
    return SKINNY_OK;
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" {

int decode_gemm_bf16(const void *x, const void *W, void *out, int M, int N, int K, void *stream) {
    return gemm_launch(x, W, out, M, N, K, stream, nullptr, 0, kWaitLimitNs);
}

int decode_gemm_bf16_ex(const void *x, const void *W, void *out, int M, int N, int K,
                        const skinny_launch_opts *opts, void *stream) {
    return gemm_launch(x, W, out, M, N, K, stream, opts, 0, kWaitLimitNs);
}

int decode_gemm_bf16_noalloc(const void *x, const void *W, void *out, int M, int N, int K,
                             void *stream) {
    return gemm_launch_static(x, W, out, M, N, K, stream);
}

int decode_gemm_bf16_reduce_rmsnorm_ex(const void *x, const void *W, void *partials, int TP,
                                       const void *residual, const void *gamma, void *out,
                                       void *residual_out, int M, int K, float eps,
                                       const skinny_launch_opts *opts, void *stream) {
    constexpr int N = SKINNY_HIDDEN;
    if (!x || !W || !partials || !gamma || !out || !residual_out) return SKINNY_ERR_NULL;
    if (M < 1 || M > SKINNY_REDUCE_MAX_M || TP < 1 || TP > SKINNY_REDUCE_MAX_TP) return SKINNY_ERR_SHAPE;
    int st = gemm_shape_ok(M, N, K);
    if (st) return st;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return SKINNY_ERR_ARG;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(partials, 16) || !aligned(gamma, 16) ||
        !aligned(out, 16) || !aligned(residual_out, 16) || (residual && !aligned(residual, 16)))
        return SKINNY_ERR_ALIGN;
    const size_t xb = static_cast<size_t>(M) * K * 2, wb = static_cast<size_t>(N) * K * 2;
    const size_t row = static_cast<size_t>(M) * N * 2, pb = row * TP, gb = N * 2;
    // Slot 0 of partials, out and residual_out are written; residual_out may be
    // residual itself (element-wise in place), nothing else may overlap.
    if (overlaps(partials, pb, x, xb) || overlaps(partials, pb, W, wb) ||
        overlaps(partials, pb, gamma, gb) || overlaps(out, row, x, xb) ||
        overlaps(out, row, W, wb) || overlaps(out, row, partials, pb) ||
        overlaps(out, row, gamma, gb) || overlaps(out, row, residual_out, row) ||
        overlaps(residual_out, row, x, xb) || overlaps(residual_out, row, W, wb) ||
        overlaps(residual_out, row, partials, pb) || overlaps(residual_out, row, gamma, gb) ||
        (residual && (overlaps(out, row, residual, row) || overlaps(partials, pb, residual, row) ||
                      (residual != residual_out && overlaps(residual_out, row, residual, row)))))
        return SKINNY_ERR_ALIAS;
    LaunchSettings ls;
    if ((st = resolve_settings(opts, &ls))) return st;
    int dev;
    if ((st = current_device(&dev))) return st;
    if ((st = check_device_pointer(x, dev)) || (st = check_device_pointer(W, dev)) ||
        (st = check_device_pointer(partials, dev)) || (st = check_device_pointer(gamma, dev)) ||
        (st = check_device_pointer(out, dev)) || (st = check_device_pointer(residual_out, dev)) ||
        (residual && (st = check_device_pointer(residual, dev))))
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceState *d = nullptr;
    if ((st = ensure_scratch(dev, s, &d))) return st;
    if ((st = pending_timeout(d))) return st;
    const GemmGeometry g = make_geometry(M, N, K, choose_ctas(N, d->sms));
    // The scratch holds two partial slots per CTA: every CTA's range must touch
    // at most two tiles, which at least one CTA per tile guarantees.
    if (g.ctas < g.tiles) return SKINNY_ERR_DEVICE;
    EncodeTiledFn enc;
    if ((st = encoder(&enc))) return st;
    const int mma_n = mma_n_for(M);
    alignas(64) CUtensorMap w_map, x_map;
    if ((st = encode_2d(enc, &w_map, W, N, K, kBlockN))) return st;
    if ((st = encode_2d(enc, &x_map, x, M, K, mma_n))) return st;
    const bool pdl = ls.pdl;
    const int l2_lead = ls.l2_lead;
    GemmArgs a = {};
    a.M = M;
    a.N = N;
    a.K = K;
    a.out = static_cast<uint16_t *>(partials);
    a.partials = d->partials;
    a.slot_floats = kSlotFloats;
    a.flags = d->flags;
    a.err = d->err;
    a.host_err = d->host_err_dev;
    a.wait_limit_ns = kWaitLimitNs;
    a.scale = 1.0f;
    a.publish_only = 1;
    a.l2_lead = l2_lead;
    a.gemm_done = d->gemm_done;
    a.clear_gemm_done = 1;
    if (launch_decode_gemm(w_map, x_map, a, mma_n, g.ctas, s, pdl, use_shallow_ring(g, pdl), dev) !=
        cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    SplitKPartials fix = {};
    fix.partials = d->partials;
    fix.slot_floats = kSlotFloats;
    fix.gemm_done = d->gemm_done;
    fix.M = M;
    fix.N = N;
    fix.K = K;
    fix.ctas = g.ctas;
    // The same CTAs per row as reduce_residual_rmsnorm: the same order of the sum
    // of squares, so out is bit-identical to the two separate calls.
    const int cpr = reduce_ctas_per_row(M, TP, residual != nullptr);
    if (launch_reduce_rmsnorm_splitk(partials, TP, residual, gamma, out, residual_out, M, eps, cpr,
                                     fix, s, pdl) != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

int decode_gemm_bf16_reduce_rmsnorm(const void *x, const void *W, void *partials, int TP,
                                    const void *residual, const void *gamma, void *out,
                                    void *residual_out, int M, int K, float eps, void *stream) {
    return decode_gemm_bf16_reduce_rmsnorm_ex(x, W, partials, TP, residual, gamma, out,
                                              residual_out, M, K, eps, nullptr, stream);
}

int decode_gemm_bf16_logits(const void *x, const void *W, void *out, int M, int N, int K,
                            int n_out, float soft_cap, float scale, void *stream) {
    if (n_out < 1 || n_out > N) return SKINNY_ERR_SHAPE;
    if (!std::isfinite(soft_cap) || !std::isfinite(scale)) return SKINNY_ERR_ARG;
    // Only the first n_out weight rows are read: the same GEMM with N = n_out.
    return gemm_launch(x, W, out, M, n_out, K, stream, nullptr, 0, kWaitLimitNs, 1,
                       soft_cap > 0.0f ? soft_cap : 0.0f, scale);
}

int decode_gemm_bf16_epilogue(const void *x, const void *W, const void *bias,
                              const void *residual, void *out, int M, int N, int K,
                              int activation, const skinny_launch_opts *opts, void *stream) {
    if (activation < SKINNY_ACT_NONE || activation > SKINNY_ACT_GELU_TANH) return SKINNY_ERR_ARG;
    Epilogue epi = {};
    epi.bias = static_cast<const uint16_t *>(bias);
    epi.residual = static_cast<const uint16_t *>(residual);
    epi.activation = activation;
    return gemm_launch(x, W, out, M, N, K, stream, opts, 0, kWaitLimitNs, 0, 0.0f, 1.0f, &epi);
}

int skinny_watchdog_selftest(const void *x, const void *W, void *out, int M, int N, int K,
                             long long timeout_ns, void *stream) {
    if (timeout_ns < 1000 || timeout_ns > 2000000000LL) return SKINNY_ERR_ARG;
    return gemm_launch(x, W, out, M, N, K, stream, nullptr, 1,
                       static_cast<unsigned long long>(timeout_ns));
}

int reduce_residual_rmsnorm_ex(const void *partials, int TP, const void *residual,
                               const void *gamma, void *out, void *residual_out, int M, float eps,
                               const skinny_launch_opts *opts, void *stream) {
    LaunchSettings ls;
    int dev, st;
    if ((st = reduce_arg_checks(partials, TP, residual, gamma, out, residual_out, M, eps)) ||
        (st = resolve_settings(opts, &ls)) ||
        (st = reduce_device_checks(partials, residual, gamma, out, residual_out, &dev)))
        return st;
    cudaError_t e = launch_reduce_rmsnorm(partials, TP, residual, gamma, out, residual_out, M, eps,
                                          reduce_ctas_per_row(M, TP, residual != nullptr),
                                          static_cast<cudaStream_t>(stream), ls.pdl);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

int skinny_reduce_selftest(const void *partials, int TP, const void *residual, const void *gamma,
                           void *out, void *residual_out, int M, float eps, long long timeout_ns,
                           void *stream) {
    if (timeout_ns < 1000 || timeout_ns > 2000000000LL) return SKINNY_ERR_ARG;
    int dev, st;
    if ((st = reduce_arg_checks(partials, TP, residual, gamma, out, residual_out, M, eps)) ||
        (st = reduce_device_checks(partials, residual, gamma, out, residual_out, &dev)))
        return st;
    cudaError_t e = launch_reduce_rmsnorm_selftest(partials, TP, residual, gamma, out,
                                                   residual_out, M, eps,
                                                   static_cast<unsigned long long>(timeout_ns),
                                                   static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

int reduce_residual_rmsnorm(const void *partials, int TP, const void *residual,
                            const void *gamma, void *out, void *residual_out, int M, float eps,
                            void *stream) {
    return reduce_residual_rmsnorm_ex(partials, TP, residual, gamma, out, residual_out, M, eps,
                                      nullptr, stream);
}

int gather_shards_bf16(const void *shards, int TP, int M, int S, void *out, void *stream) {
    if (!shards || !out) return SKINNY_ERR_NULL;
    if (TP < 1 || TP > SKINNY_GATHER_MAX_TP || M < 1 || M > SKINNY_GATHER_MAX_M || S < 8 ||
        (S % 8) != 0 || static_cast<long long>(TP) * S > (1LL << 30))
        return SKINNY_ERR_SHAPE;
    if (!aligned(shards, 16) || !aligned(out, 16)) return SKINNY_ERR_ALIGN;
    const size_t bytes = static_cast<size_t>(TP) * M * S * 2;
    if (overlaps(out, bytes, shards, bytes)) return SKINNY_ERR_ALIAS;
    int dev, st;
    if ((st = current_device(&dev))) return st;
    DeviceState *d = nullptr;
    if ((st = device_state(dev, &d))) return st;
    if ((st = check_device_pointer(shards, dev)) || (st = check_device_pointer(out, dev))) return st;
    bool pdl;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        pdl = g_pdl;
    }
    if (launch_gather(shards, TP, M, S, out, static_cast<cudaStream_t>(stream), pdl) != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

int qk_norm_rope_bf16(const skinny_qk_norm_rope_args *p, const skinny_launch_opts *opts,
                      void *stream) {
    if (!p) return SKINNY_ERR_NULL;
    const skinny_kv_cache *cache = &p->cache;
    const bool has_cache = cache->k || cache->v;
    if (!p->qkv || !p->q_out || (p->rot_dim != 0 && (!p->rope || !p->positions)) ||
        (has_cache && !p->slots))
        return SKINNY_ERR_NULL;
    const int D = p->head_dim;
    constexpr int kMaxRows = 1 << 30;  // the kernel looks two of its rounds ahead in 32 bits
    if (p->M < 1 || p->M > kMaxRows || p->q_heads < 1 || p->q_heads > kMaxHeads || p->kv_heads < 1 ||
        p->kv_heads > kMaxHeads || D < 8 || D > kMaxHeadDim || D % 8 != 0 || p->rot_dim < 0 ||
        p->rot_dim > D || p->rot_dim % 16 != 0 || (p->rot_dim > 0 && p->max_pos < 1))
        return SKINNY_ERR_SHAPE;
    const long long q_width = static_cast<long long>(p->q_heads) * D;
    const long long kv_width = static_cast<long long>(p->kv_heads) * D;
    const long long width = q_width + 2 * kv_width;
    constexpr long long kMaxStride = 1ll << 30;  // rows * stride stays far below 2^63 bytes
    if (p->qkv_stride < width || p->qkv_stride > kMaxStride || p->q_stride < q_width ||
        p->q_stride > kMaxStride || (p->k_out && (p->k_stride < kv_width || p->k_stride > kMaxStride)))
        return SKINNY_ERR_SHAPE;
    if (!(p->eps > 0.0f) || !std::isfinite(p->eps) || p->interleaved < 0 || p->interleaved > 1)
        return SKINNY_ERR_ARG;
    if (!aligned(p->qkv, 16) || !aligned(p->q_out, 16) || !aligned(p->k_out, 16) ||
        !aligned(p->q_gamma, 16) || !aligned(p->k_gamma, 16) || !aligned(p->rope, 16) ||
        !aligned(p->positions, 4) || !aligned(p->slots, 8) || p->qkv_stride % 8 != 0 ||
        p->q_stride % 8 != 0 || (p->k_out && p->k_stride % 8 != 0))
        return SKINNY_ERR_ALIGN;
    int st;
    size_t pool = 0;
    if (has_cache) {
        if (cache->kv_heads != p->kv_heads || cache->head_dim != D) return SKINNY_ERR_SHAPE;
        if ((st = check_cache(cache, true, &pool))) return st;
    }
    // Every output against every input and the other outputs; q_out and k_out may be
    // their own heads of qkv in place. One row has no distance to a next one: its strides
    // need not agree (a view of a single row has its own width there).
    const struct { const void *p; size_t n; } in[] = {
        {p->qkv, row_span(p->M, p->qkv_stride, width)},
        {p->q_gamma, static_cast<size_t>(D) * 2},
        {p->k_gamma, static_cast<size_t>(D) * 2},
        {p->rot_dim ? p->rope : nullptr, static_cast<size_t>(p->max_pos) * p->rot_dim * 4},
        {p->rot_dim ? p->positions : nullptr, static_cast<size_t>(p->M) * 4},
        {has_cache ? p->slots : nullptr, static_cast<size_t>(p->M) * 8}};
    const bool q_in_place = p->q_out == p->qkv && (p->M == 1 || p->q_stride == p->qkv_stride);
    const bool k_in_place = p->k_out == static_cast<const uint16_t *>(p->qkv) + q_width &&
                            (p->M == 1 || p->k_stride == p->qkv_stride);
    const struct { const void *p; size_t n; bool in_place; } outs[] = {
        {p->q_out, row_span(p->M, p->q_stride, q_width), q_in_place},
        {p->k_out, p->k_out ? row_span(p->M, p->k_stride, kv_width) : 0, k_in_place},
        {has_cache ? cache->k : nullptr, pool, false},
        {has_cache ? cache->v : nullptr, pool, false}};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i].p) continue;
        for (int j = 0; j < 6; ++j)
            if (in[j].p && !(j == 0 && outs[i].in_place) && overlaps(outs[i].p, outs[i].n, in[j].p, in[j].n))
                return SKINNY_ERR_ALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (outs[j].p && !(outs[i].in_place && outs[j].in_place) && !(i == 2 && j == 3) &&
                overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return SKINNY_ERR_ALIAS;
    }
    LaunchSettings ls;
    if ((st = resolve_settings(opts, &ls))) return st;
    int dev;
    if ((st = current_device(&dev))) return st;
    DeviceState *d = nullptr;
    if ((st = device_state(dev, &d))) return st;
    for (const auto &b : in)
        if (b.p && (st = check_device_pointer(b.p, dev))) return st;
    for (const auto &b : outs)
        if (b.p && !b.in_place && (st = check_device_pointer(b.p, dev))) return st;
    RopeArgs a = {};
    a.qkv = static_cast<const uint16_t *>(p->qkv);
    a.qkv_stride = p->qkv_stride;
    a.rows = p->M;
    a.q_heads = p->q_heads;
    a.kv_heads = p->kv_heads;
    a.head_dim = D;
    a.q_gamma = static_cast<const uint16_t *>(p->q_gamma);
    a.k_gamma = static_cast<const uint16_t *>(p->k_gamma);
    a.eps = p->eps;
    a.inv_dim = 1.0f / static_cast<float>(D);
    a.rope = static_cast<const float *>(p->rope);
    a.max_pos = p->max_pos;
    a.rot_dim = p->rot_dim;
    a.interleaved = p->interleaved;
    a.positions = static_cast<const int *>(p->positions);
    a.q_out = static_cast<uint16_t *>(p->q_out);
    a.q_stride = p->q_stride;
    a.k_out = static_cast<uint16_t *>(p->k_out);
    a.k_stride = p->k_stride;
    if (has_cache) {
        a.k_cache = static_cast<uint16_t *>(cache->k);
        a.v_cache = static_cast<uint16_t *>(cache->v);
        a.page_size = cache->page_size;
        a.page_shift = log2_or_minus_one(cache->page_size);
        a.num_slots = static_cast<long long>(cache->num_pages) * cache->page_size;
        a.page_stride = cache->page_stride;
        a.token_stride = cache->token_stride;
        a.head_stride = cache->head_stride;
        a.slots = static_cast<const long long *>(p->slots);
    }
    if (launch_qk_norm_rope(a, d->sms, static_cast<cudaStream_t>(stream), ls.pdl) != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

size_t skinny_attention_workspace_bytes(int num_sms) {
    return num_sms < 1 ? 0 : attn_workspace_bytes(attn_sms(num_sms));
}

int decode_attention_bf16(const skinny_decode_attention_args *p, const skinny_launch_opts *opts,
                          void *stream) {
    if (!p || !p->q || !p->block_table || !p->lengths || !p->out || !p->workspace)
        return SKINNY_ERR_NULL;
    const skinny_kv_cache *c = &p->cache;
    size_t pool = 0;
    int st = check_cache(c, false, &pool);
    if (st) return st;
    const int D = c->head_dim;
    if (D != 64 && D != 96 && D != 128 && D != 192 && D != 256) return SKINNY_ERR_SHAPE;
    if (p->rows < 1 || p->rows > SKINNY_ATTENTION_MAX_ROWS || p->q_heads < 1 ||
        p->q_heads > kMaxHeads || p->q_heads % c->kv_heads != 0 || p->table_width < 1 ||
        p->table_stride < p->table_width || p->table_stride > (1ll << 40))
        return SKINNY_ERR_SHAPE;
    const long long capacity = static_cast<long long>(p->table_width) * c->page_size;
    if (capacity >= (1ll << 30)) return SKINNY_ERR_SHAPE;
    const int group = p->q_heads / c->kv_heads, most = 8 * attn_max_nb(D);
    const int head_blocks = (group + most - 1) / most;
    const long long tiles = (capacity + kAttnMinTile - 1) / kAttnMinTile;
    if (tiles * p->rows * c->kv_heads * head_blocks >= (1ll << 31)) return SKINNY_ERR_SHAPE;
    const long long q_width = static_cast<long long>(p->q_heads) * D;
    if (p->q_stride < q_width || p->q_stride > (1ll << 30)) return SKINNY_ERR_SHAPE;
    if (p->window < 0 || p->sinks < 0 || !std::isfinite(p->scale)) return SKINNY_ERR_ARG;
    if (!aligned(p->q, 16) || !aligned(p->out, 16) || !aligned(p->workspace, 16) ||
        !aligned(p->block_table, 4) || !aligned(p->lengths, 4) || !aligned(p->lse, 4) ||
        p->q_stride % 8 != 0)
        return SKINNY_ERR_ALIGN;
    const size_t heads = static_cast<size_t>(p->rows) * p->q_heads;
    const struct { const void *p; size_t n; } in[] = {
        {p->q, row_span(p->rows, p->q_stride, q_width)}, {c->k, pool}, {c->v, pool},
        {p->block_table, (static_cast<size_t>(p->rows - 1) * p->table_stride + p->table_width) * 4},
        {p->lengths, static_cast<size_t>(p->rows) * 4}};
    const struct { const void *p; size_t n; } outs[] = {
        {p->out, heads * D * 2}, {p->lse, heads * 4}, {p->workspace, p->workspace_bytes}};
    for (int i = 0; i < 3; ++i) {
        if (!outs[i].p) continue;
        for (const auto &b : in)
            if (overlaps(outs[i].p, outs[i].n, b.p, b.n)) return SKINNY_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (outs[j].p && overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SKINNY_ERR_ALIAS;
    }
    LaunchSettings ls;
    if ((st = resolve_settings(opts, &ls))) return st;
    int dev;
    if ((st = current_device(&dev))) return st;
    DeviceState *d = nullptr;
    if ((st = device_state(dev, &d))) return st;
    const int sms = attn_sms(d->sms);
    if (p->workspace_bytes < attn_workspace_bytes(sms)) return SKINNY_ERR_SHAPE;
    for (const auto &b : in)
        if ((st = check_device_pointer(b.p, dev))) return st;
    for (const auto &b : outs)
        if (b.p && (st = check_device_pointer(b.p, dev))) return st;
    AttentionArgs a = {};
    a.q = static_cast<const uint16_t *>(p->q);
    a.q_stride = p->q_stride;
    a.k = static_cast<const uint16_t *>(c->k);
    a.v = static_cast<const uint16_t *>(c->v);
    a.num_pages = c->num_pages;
    a.page_size = c->page_size;
    a.page_shift = log2_or_minus_one(c->page_size);
    a.page_stride = c->page_stride;
    a.token_stride = c->token_stride;
    a.head_stride = c->head_stride;
    a.block_table = static_cast<const int *>(p->block_table);
    a.table_stride = p->table_stride;
    a.lengths = static_cast<const int *>(p->lengths);
    a.rows = p->rows;
    a.q_heads = p->q_heads;
    a.kv_heads = c->kv_heads;
    a.group = group;
    a.head_blocks = head_blocks;
    a.block_heads = (group + head_blocks - 1) / head_blocks;
    a.capacity = static_cast<int>(capacity);
    a.wide = pool > (1ull << 36);
    a.window = p->window;
    a.sinks = p->sinks;
    a.scale_log2 = p->scale * 1.44269504088896341f;
    a.out = static_cast<uint16_t *>(p->out);
    a.lse = static_cast<float *>(p->lse);
    a.counters = static_cast<unsigned *>(p->workspace);
    static_assert(kAttnCounterBytes == SKINNY_ATTENTION_COUNTER_BYTES, "the header's number");
    a.partials = reinterpret_cast<float *>(static_cast<char *>(p->workspace) + kAttnCounterBytes);
    if (launch_decode_attention(a, D, sms, dev, static_cast<cudaStream_t>(stream), ls.pdl) !=
        cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_LAUNCH;
    }
    return SKINNY_OK;
}

const char *skinny_status_string(int status) {
    switch (status) {
        case SKINNY_OK: return "ok";
        case SKINNY_ERR_NULL: return "a required pointer is NULL";
        case SKINNY_ERR_SHAPE: return "a size is outside the accepted range";
        case SKINNY_ERR_ALIGN: return "a pointer is not aligned as required";
        case SKINNY_ERR_DEVICE: return "no sm_103 device, or a pointer is not memory of the current device";
        case SKINNY_ERR_LAUNCH: return "the CUDA launch failed";
        case SKINNY_ERR_ALIAS: return "an output overlaps an input or the other output";
        case SKINNY_ERR_CAPTURE: return "first call on this device made during stream capture";
        case SKINNY_ERR_ALLOC: return "scratch allocation failed";
        case SKINNY_ERR_TIMEOUT: return "a kernel's bounded internal wait ran out";
        case SKINNY_ERR_ARG: return "a scalar argument is invalid";
        case SKINNY_ERR_INDEX: return "a kernel met an index out of range in device memory";
        default: return "unknown status";
    }
}

int skinny_device_error(int device, int *word) {
    if (device < 0 || device >= kMaxDevices) return SKINNY_ERR_DEVICE;
    if (word) *word = 0;
    int prev = -1;
    if (cudaGetDevice(&prev) != cudaSuccess) {
        cudaGetLastError();
        return SKINNY_ERR_DEVICE;
    }
    if (cudaSetDevice(device) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        cudaSetDevice(prev);
        return SKINNY_ERR_DEVICE;
    }
    int value = 0;
    int st = SKINNY_OK;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        DeviceState &d = g_devices[device];
        if (d.scratch) {
            if (cudaMemcpy(&value, d.err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) {
                cudaGetLastError();
                st = SKINNY_ERR_DEVICE;
            } else if (value != 0 || *reinterpret_cast<volatile int *>(d.host_err) != 0) {
                // A kernel gave up part-way: clear the words and the partial flags,
                // which lets later calls run again.
                if (cudaMemset(d.err, 0, sizeof(int)) != cudaSuccess ||
                    cudaMemset(d.flags, 0, d.flag_bytes) != cudaSuccess) {
                    cudaGetLastError();
                    st = SKINNY_ERR_DEVICE;
                } else {
                    if (value == 0) value = kErrUnknown;
                    *reinterpret_cast<volatile int *>(d.host_err) = 0;
                }
            }
        }
    }
    // The reduce kernel's own word (its cluster exchange waits).
    int reduce_word = 0;
    if (st == SKINNY_OK && reduce_error_word(&reduce_word, true) != cudaSuccess) {
        cudaGetLastError();
        st = SKINNY_ERR_DEVICE;
    }
    if (reduce_word) value |= kErrReduceExchange;
    // The words of the kernels that read indices from device memory.
    int rope_word = 0, attention_word = 0;
    if (st == SKINNY_OK && (rope_error_word(&rope_word, true) != cudaSuccess ||
                            attention_error_word(&attention_word, true) != cudaSuccess)) {
        cudaGetLastError();
        st = SKINNY_ERR_DEVICE;
    }
    if (rope_word || attention_word) value |= kErrIndex;
    cudaSetDevice(prev);
    if (word) *word = value;
    if (st != SKINNY_OK) return st;
    if (value == kErrIndex) return SKINNY_ERR_INDEX;
    return value ? SKINNY_ERR_TIMEOUT : SKINNY_OK;
}

int skinny_set_pdl(int enable) {
    std::lock_guard<std::mutex> lock(g_mutex);
    const int prev = g_pdl ? 1 : 0;
    g_pdl = enable != 0;
    return prev;
}

int skinny_set_l2_prefetch(int blocks) {
    if (blocks < 0 || blocks > kL2LeadMax) return -1;
    std::lock_guard<std::mutex> lock(g_mutex);
    const int prev = g_l2_lead;
    g_l2_lead = blocks;
    return prev;
}

int skinny_gemm_plan_query(int M, int N, int K, int num_sms, skinny_gemm_plan *plan) {
    if (!plan) return SKINNY_ERR_NULL;
    if (num_sms < 1) return SKINNY_ERR_ARG;
    int st = gemm_shape_ok(M, N, K);
    if (st) return st;
    const GemmGeometry g = make_geometry(M, N, K, choose_ctas(N, num_sms));
    plan->tiles = g.tiles;
    plan->kblocks = g.kblocks;
    plan->blocks = g.blocks;
    plan->ctas = g.ctas;
    plan->mma_n = mma_n_for(M);
    bool pdl;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        pdl = g_pdl;
    }
    plan->stages = gemm_stages(plan->mma_n, use_shallow_ring(g, pdl));
    plan->smem_bytes = gemm_smem_bytes(plan->mma_n, use_shallow_ring(g, pdl));
    int split = 0;
    for (int t = 0; t < g.tiles; ++t) {
        int first, last;
        tile_contributors(g, t, first, last);
        split += first != last;
    }
    plan->split_tiles = split;
    return SKINNY_OK;
}

int skinny_gemm_cta_pieces(int M, int N, int K, int num_sms, int cta, int *tile, int *kb0,
                           int *kb1, int *slot, int max_pieces) {
    if (!tile || !kb0 || !kb1 || !slot || num_sms < 1 || gemm_shape_ok(M, N, K)) return -1;
    const GemmGeometry g = make_geometry(M, N, K, choose_ctas(N, num_sms));
    if (cta < 0 || cta >= g.ctas) return -1;
    const int r = range_of_block(g, cta);
    const int n = cta_piece_count(g, r);
    for (int q = 0; q < n && q < max_pieces; ++q) {
        const Piece p = cta_piece(g, r, q);
        tile[q] = p.tile;
        kb0[q] = p.kb0;
        kb1[q] = p.kb1;
        const bool whole = p.kb0 == 0 && p.kb1 == g.kblocks;
        slot[q] = whole ? -1 : partial_slot(g, r, p.tile);
    }
    return n;
}

}  // extern "C"
