"""Python binding of libskinny.so (include/skinny.h): argument marshalling only.

Every computation runs in the library's CUDA kernels; this module checks that
PyTorch tensors have the shapes and dtypes the C ABI documents, passes their
device pointers and the current CUDA stream, and turns nonzero status codes into
``SkinnyError``. There is no fallback: if the library is missing, importing the
operations raises.

    decode_gemm_bf16(x, W, out)                      out = x @ W^T (BF16)
    reduce_residual_rmsnorm(partials, residual, gamma, out, residual_out, eps)
    gather_shards_bf16(shards, out)                  TP shards side by side
    decode_gemm_bf16_epilogue(x, W, out, bias, activation, residual)
                                                     out = act(x @ W^T + bias) + residual
    decode_gemm_bf16_lora(x, W, out, A, B, adapters, ...)
                                                     the same with an adapter for each row
    qk_norm_rope_bf16(qkv, ...)                      per-head norm, rotation, cache append
    decode_attention_bf16(q, k_cache, v_cache, ...)  one token per row over a paged cache
    decode_attention_shared_prefix_bf16(q, k_cache, v_cache, ...)
                                                     the same behind a prefix all rows share
    token_logprobs_bf16(logits, tokens, logprobs, ...)
                                                     log probabilities, entropy, top tokens
"""
import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "libskinny.so")
HIDDEN = 7168
GEMM_MAX_M = 64
REDUCE_MAX_M = 64
REDUCE_MAX_TP = 8

STATUS = {
    0: "SKINNY_OK", 1: "SKINNY_ERR_NULL", 2: "SKINNY_ERR_SHAPE", 3: "SKINNY_ERR_ALIGN",
    4: "SKINNY_ERR_DEVICE", 5: "SKINNY_ERR_LAUNCH", 6: "SKINNY_ERR_ALIAS",
    7: "SKINNY_ERR_CAPTURE", 8: "SKINNY_ERR_ALLOC", 9: "SKINNY_ERR_TIMEOUT",
    10: "SKINNY_ERR_ARG", 11: "SKINNY_ERR_INDEX",
}


class SkinnyError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


class LaunchOpts(ctypes.Structure):
    """skinny_launch_opts: per-call settings, -1 = the process-wide one (for
    l2_after_reduce: off)."""
    _fields_ = [("pdl", ctypes.c_int), ("l2_prefetch", ctypes.c_int),
                ("l2_after_reduce", ctypes.c_int)]


def _opts(pdl, l2_prefetch, l2_after_reduce=None):
    """A LaunchOpts for the given keywords, or None if all are None (the call
    then goes to the plain entry point and the process-wide settings)."""
    if pdl is None and l2_prefetch is None and l2_after_reduce is None:
        return None
    return LaunchOpts(-1 if pdl is None else int(bool(pdl)),
                      -1 if l2_prefetch is None else int(l2_prefetch),
                      -1 if l2_after_reduce is None else int(l2_after_reduce))


class GemmPlan(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_int), ("kblocks", ctypes.c_int),
                ("blocks", ctypes.c_longlong), ("ctas", ctypes.c_int),
                ("mma_n", ctypes.c_int), ("stages", ctypes.c_int),
                ("smem_bytes", ctypes.c_int), ("split_tiles", ctypes.c_int)]


class KVCacheArgs(ctypes.Structure):
    """skinny_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_stride", ctypes.c_longlong),
                ("token_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


class QkNormRopeArgs(ctypes.Structure):
    """skinny_qk_norm_rope_args."""
    _fields_ = [("qkv", ctypes.c_void_p), ("qkv_stride", ctypes.c_longlong), ("M", ctypes.c_int),
                ("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("q_gamma", ctypes.c_void_p), ("k_gamma", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("rope", ctypes.c_void_p), ("max_pos", ctypes.c_int),
                ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("positions", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("q_stride", ctypes.c_longlong), ("k_out", ctypes.c_void_p),
                ("k_stride", ctypes.c_longlong), ("cache", KVCacheArgs),
                ("slots", ctypes.c_void_p)]


class SharedPrefixAttentionArgs(ctypes.Structure):
    """skinny_shared_prefix_attention_args."""
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_longlong), ("rows", ctypes.c_int),
                ("q_heads", ctypes.c_int), ("cache", KVCacheArgs),
                ("prefix_table", ctypes.c_void_p), ("prefix_width", ctypes.c_int),
                ("prefix_length", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_longlong), ("table_width", ctypes.c_int),
                ("lengths", ctypes.c_void_p), ("scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class LoraArgs(ctypes.Structure):
    """skinny_lora."""
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("adapters", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("num_adapters", ctypes.c_int), ("rank", ctypes.c_int)]


class TokenLogprobsArgs(ctypes.Structure):
    """skinny_token_logprobs_args."""
    _fields_ = [("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_longlong),
                ("M", ctypes.c_int), ("V", ctypes.c_int), ("tokens", ctypes.c_void_p),
                ("given", ctypes.c_int), ("logprobs", ctypes.c_void_p),
                ("entropy", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("top", ctypes.c_int),
                ("top_logprobs", ctypes.c_void_p), ("top_tokens", ctypes.c_void_p)]


class DecodeAttentionArgs(ctypes.Structure):
    """skinny_decode_attention_args."""
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_longlong), ("rows", ctypes.c_int),
                ("q_heads", ctypes.c_int), ("cache", KVCacheArgs),
                ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_longlong),
                ("table_width", ctypes.c_int), ("lengths", ctypes.c_void_p),
                ("window", ctypes.c_int), ("sinks", ctypes.c_int), ("scale", ctypes.c_float),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


# The same structures as one packed string each: a third of the host time of
# filling a ctypes.Structure field by field.
_CACHE = "PPiiiiqqq"
_pack_rope = struct.Struct("@PqiiiiPPfPiiiPPqPq" + _CACHE + "P").pack
_pack_attention = struct.Struct("@Pqii" + _CACHE + "PqiPiifPPPN").pack
_pack_prefix = struct.Struct("@Pqii" + _CACHE + "PiPPqiPfPPPN").pack
_pack_logprobs = struct.Struct("@PqiiPiPPPiPP").pack
_pack_lora = struct.Struct("@PPPPii").pack
_NO_CACHE = (0,) * 9


_lib = None


def load_library(path: str = LIBRARY):
    """Load libskinny.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"{path} is missing: build it with "
                      "`python -m skinny_bf16_gemm_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    op = ctypes.POINTER(LaunchOpts)
    lib.decode_gemm_bf16.argtypes = [vp, vp, vp, i32, i32, i32, vp]
    lib.decode_gemm_bf16.restype = i32
    lib.decode_gemm_bf16_ex.argtypes = [vp, vp, vp, i32, i32, i32, op, vp]
    lib.decode_gemm_bf16_ex.restype = i32
    lib.reduce_residual_rmsnorm.argtypes = [vp, i32, vp, vp, vp, vp, i32, f32, vp]
    lib.reduce_residual_rmsnorm.restype = i32
    lib.reduce_residual_rmsnorm_ex.argtypes = [vp, i32, vp, vp, vp, vp, i32, f32, op, vp]
    lib.reduce_residual_rmsnorm_ex.restype = i32
    lib.decode_gemm_bf16_logits.argtypes = [vp, vp, vp, i32, i32, i32, i32, f32, f32, vp]
    lib.decode_gemm_bf16_logits.restype = i32
    lib.decode_gemm_bf16_epilogue.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, op, vp]
    lib.decode_gemm_bf16_epilogue.restype = i32
    lib.decode_gemm_bf16_lora.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, op, vp]
    lib.decode_gemm_bf16_lora.restype = i32
    lib.decode_gemm_bf16_reduce_rmsnorm.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i32,
                                                    f32, vp]
    lib.decode_gemm_bf16_reduce_rmsnorm.restype = i32
    lib.decode_gemm_bf16_reduce_rmsnorm_ex.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i32,
                                                       f32, op, vp]
    lib.decode_gemm_bf16_reduce_rmsnorm_ex.restype = i32
    lib.qk_norm_rope_bf16.argtypes = [vp, op, vp]
    lib.qk_norm_rope_bf16.restype = i32
    lib.decode_attention_bf16.argtypes = [vp, op, vp]
    lib.decode_attention_bf16.restype = i32
    lib.token_logprobs_bf16.argtypes = [vp, op, vp]
    lib.token_logprobs_bf16.restype = i32
    lib.decode_attention_shared_prefix_bf16.argtypes = [vp, op, vp]
    lib.decode_attention_shared_prefix_bf16.restype = i32
    lib.skinny_shared_prefix_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.skinny_shared_prefix_workspace_bytes.restype = ctypes.c_size_t
    lib.skinny_attention_workspace_bytes.argtypes = [i32]
    lib.skinny_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.gather_shards_bf16.argtypes = [vp, i32, i32, i32, vp, vp]
    lib.gather_shards_bf16.restype = i32
    lib.skinny_status_string.argtypes = [i32]
    lib.skinny_status_string.restype = ctypes.c_char_p
    lib.skinny_device_error.argtypes = [i32, ctypes.POINTER(i32)]
    lib.skinny_device_error.restype = i32
    lib.skinny_set_pdl.argtypes = [i32]
    lib.skinny_set_pdl.restype = i32
    lib.skinny_set_l2_prefetch.argtypes = [i32]
    lib.skinny_set_l2_prefetch.restype = i32
    lib.skinny_gemm_plan_query.argtypes = [i32, i32, i32, i32, ctypes.POINTER(GemmPlan)]
    lib.skinny_gemm_plan_query.restype = i32
    ip = ctypes.POINTER(i32)
    lib.skinny_gemm_cta_pieces.argtypes = [i32, i32, i32, i32, i32, ip, ip, ip, ip, i32]
    lib.skinny_gemm_cta_pieces.restype = i32
    lib.skinny_watchdog_selftest.argtypes = [vp, vp, vp, i32, i32, i32, ctypes.c_longlong, vp]
    lib.skinny_watchdog_selftest.restype = i32
    lib.skinny_reduce_selftest.argtypes = [vp, i32, vp, vp, vp, vp, i32, f32, ctypes.c_longlong, vp]
    lib.skinny_reduce_selftest.restype = i32
    lib.skinny_shared_prefix_selftest.argtypes = [vp, ctypes.c_longlong, vp]
    lib.skinny_shared_prefix_selftest.restype = i32
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().skinny_status_string(int(status)).decode()


def _stream_handle(stream):
    import torch
    if stream is None:
        # torch.cuda.current_stream() without the Stream object it makes (3 us a call).
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(status: int, where: str):
    if status != 0:
        raise SkinnyError(status, where)


def _bf16_cuda(t, name, shape=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor (got {t.dtype} on {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def decode_gemm_bf16(x, W, out, stream=None, pdl=None, l2_prefetch=None, l2_after_reduce=None):
    """out[M, N] = x[M, K] @ W[N, K]^T on the current (or given) stream.

    x, W, out: contiguous CUDA bfloat16 tensors. Returns ``out``. pdl and
    l2_prefetch, when given, are this call's launch settings (decode_gemm_bf16_ex)
    instead of the process-wide ones; l2_after_reduce (weight blocks, 0..64) is
    for a call right behind decode_gemm_bf16_reduce_rmsnorm (see skinny.h).
    """
    _bf16_cuda(x, "x")
    _bf16_cuda(W, "W")
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} and W {tuple(W.shape)} must be [M,K] and [N,K]")
    M, K = x.shape
    N = W.shape[0]
    _bf16_cuda(out, "out", (M, N))
    o = _opts(pdl, l2_prefetch, l2_after_reduce)
    lib = load_library()
    if o is None:
        st = lib.decode_gemm_bf16(x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K,
                                  _stream_handle(stream))
    else:
        st = lib.decode_gemm_bf16_ex(x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K,
                                     ctypes.byref(o), _stream_handle(stream))
    _check(st, "decode_gemm_bf16")
    return out


def decode_gemm_bf16_logits(x, W, out, soft_cap=0.0, scale=1.0, stream=None):
    """lm_head logits out[M, n_out] = scale * cap * tanh((x @ W[:n_out]^T) / cap)
    (no tanh if soft_cap <= 0); n_out = out.shape[1] <= W.shape[0]. Returns out."""
    _bf16_cuda(x, "x")
    _bf16_cuda(W, "W")
    _bf16_cuda(out, "out")
    if x.dim() != 2 or W.dim() != 2 or out.dim() != 2 or x.shape[1] != W.shape[1] \
            or out.shape[0] != x.shape[0]:
        raise ValueError("x [M,K], W [N,K] and out [M,n_out] do not fit together")
    M, K = x.shape
    N, n_out = W.shape[0], out.shape[1]
    st = load_library().decode_gemm_bf16_logits(x.data_ptr(), W.data_ptr(), out.data_ptr(), M,
                                                N, K, n_out, float(soft_cap), float(scale),
                                                _stream_handle(stream))
    _check(st, "decode_gemm_bf16_logits")
    return out


ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def decode_gemm_bf16_epilogue(x, W, out, bias=None, activation="none", residual=None, stream=None,
                              pdl=None, l2_prefetch=None):
    """out[M, N] = act(x[M, K] @ W[N, K]^T + bias[N]) + residual[M, N].

    bias and residual may be None; residual may be out itself. activation: one of
    ACTIVATIONS. FP32 throughout, one BF16 rounding. x, W, out, pdl and l2_prefetch
    as for decode_gemm_bf16. Returns ``out``.
    """
    _bf16_cuda(x, "x")
    _bf16_cuda(W, "W")
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} and W {tuple(W.shape)} must be [M,K] and [N,K]")
    M, K = x.shape
    N = W.shape[0]
    _bf16_cuda(out, "out", (M, N))
    if bias is not None:
        _bf16_cuda(bias, "bias", (N,))
    if residual is not None:
        _bf16_cuda(residual, "residual", (M, N))
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    o = _opts(pdl, l2_prefetch)
    st = load_library().decode_gemm_bf16_epilogue(
        x.data_ptr(), W.data_ptr(), None if bias is None else bias.data_ptr(),
        None if residual is None else residual.data_ptr(), out.data_ptr(), M, N, K, act,
        None if o is None else ctypes.byref(o), _stream_handle(stream))
    _check(st, "decode_gemm_bf16_epilogue")
    return out


def decode_gemm_bf16_lora(x, W, out, A, B, adapters, scales=None, bias=None, activation="none",
                          residual=None, stream=None, pdl=None, l2_prefetch=None):
    """out[M, N] = act(x @ W^T + c_a (x @ A_a^T) @ B_a^T + bias) + residual, a = adapters[m].

    A [num_adapters, rank, K] and B [num_adapters, N, rank], contiguous CUDA bfloat16;
    adapters [M] int32 (negative: the row has none); scales [num_adapters] FP32 or None (1).
    rank: a multiple of 8 up to 128. The rest as for decode_gemm_bf16_epilogue. Returns ``out``.
    """
    import torch
    _bf16_cuda(x, "x")
    _bf16_cuda(W, "W")
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} and W {tuple(W.shape)} must be [M,K] and [N,K]")
    M, K = x.shape
    N = W.shape[0]
    _bf16_cuda(out, "out", (M, N))
    _bf16_cuda(A, "A")
    if A.dim() != 3 or A.shape[2] != K:
        raise ValueError(f"A must be [num_adapters, rank, {K}], got {tuple(A.shape)}")
    count, rank = A.shape[:2]
    _bf16_cuda(B, "B", (count, N, rank))
    adapters_ptr = _plain_cuda(adapters, "adapters", torch.int32, (M,))
    scales_ptr = 0 if scales is None else _plain_cuda(scales, "scales", torch.float32, (count,))
    if bias is not None:
        _bf16_cuda(bias, "bias", (N,))
    if residual is not None:
        _bf16_cuda(residual, "residual", (M, N))
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    o = _opts(pdl, l2_prefetch)
    st = load_library().decode_gemm_bf16_lora(
        x.data_ptr(), W.data_ptr(), _pack_lora(A.data_ptr(), B.data_ptr(), adapters_ptr, scales_ptr, count, rank),
        None if bias is None else bias.data_ptr(), None if residual is None else residual.data_ptr(),
        out.data_ptr(), M, N, K, act, None if o is None else ctypes.byref(o), _stream_handle(stream))
    _check(st, "decode_gemm_bf16_lora")
    return out


def reduce_residual_rmsnorm(partials, residual, gamma, out, residual_out, eps=1e-6,
                            stream=None, pdl=None):
    """(out, residual_out) of the rank-order reduce + residual + RMSNorm.

    partials [TP, M, 7168], residual [M, 7168] or None, gamma [7168],
    out and residual_out [M, 7168]; all contiguous CUDA bfloat16. pdl, when
    given, is this call's setting (reduce_residual_rmsnorm_ex).
    """
    _bf16_cuda(partials, "partials")
    if partials.dim() != 3 or partials.shape[2] != HIDDEN:
        raise ValueError(f"partials must be [TP, M, {HIDDEN}], got {tuple(partials.shape)}")
    TP, M, _ = partials.shape
    if residual is not None:
        _bf16_cuda(residual, "residual", (M, HIDDEN))
    _bf16_cuda(gamma, "gamma", (HIDDEN,))
    _bf16_cuda(out, "out", (M, HIDDEN))
    _bf16_cuda(residual_out, "residual_out", (M, HIDDEN))
    args = (partials.data_ptr(), TP, None if residual is None else residual.data_ptr(),
            gamma.data_ptr(), out.data_ptr(), residual_out.data_ptr(), M, float(eps))
    o = _opts(pdl, None)
    if o is None:
        st = load_library().reduce_residual_rmsnorm(*args, _stream_handle(stream))
    else:
        st = load_library().reduce_residual_rmsnorm_ex(*args, ctypes.byref(o),
                                                       _stream_handle(stream))
    _check(st, "reduce_residual_rmsnorm")
    return out, residual_out


def decode_gemm_bf16_reduce_rmsnorm(x, W, partials, residual, gamma, out, residual_out,
                                    eps=1e-6, stream=None, pdl=None, l2_prefetch=None):
    """The row-parallel linear with the reduce + residual + RMSNorm after it.

    x [M, K], W [7168, K]; partials [TP, M, 7168] (slot 0 receives x @ W^T,
    slots 1.. are read); residual [M, 7168] or None; gamma [7168]; out and
    residual_out [M, 7168]; all contiguous CUDA bfloat16. Returns
    (out, residual_out), bit for bit those of decode_gemm_bf16 followed by
    reduce_residual_rmsnorm. pdl and l2_prefetch as for decode_gemm_bf16.
    """
    _bf16_cuda(x, "x")
    _bf16_cuda(W, "W")
    _bf16_cuda(partials, "partials")
    if x.dim() != 2 or W.dim() != 2 or tuple(W.shape) != (HIDDEN, x.shape[1]):
        raise ValueError(f"x must be [M, K] and W [{HIDDEN}, K]")
    M, K = x.shape
    if partials.dim() != 3 or tuple(partials.shape[1:]) != (M, HIDDEN):
        raise ValueError(f"partials must be [TP, {M}, {HIDDEN}], got {tuple(partials.shape)}")
    TP = partials.shape[0]
    if residual is not None:
        _bf16_cuda(residual, "residual", (M, HIDDEN))
    _bf16_cuda(gamma, "gamma", (HIDDEN,))
    _bf16_cuda(out, "out", (M, HIDDEN))
    _bf16_cuda(residual_out, "residual_out", (M, HIDDEN))
    args = (x.data_ptr(), W.data_ptr(), partials.data_ptr(), TP,
            None if residual is None else residual.data_ptr(), gamma.data_ptr(), out.data_ptr(),
            residual_out.data_ptr(), M, K, float(eps))
    o = _opts(pdl, l2_prefetch)
    if o is None:
        st = load_library().decode_gemm_bf16_reduce_rmsnorm(*args, _stream_handle(stream))
    else:
        st = load_library().decode_gemm_bf16_reduce_rmsnorm_ex(*args, ctypes.byref(o),
                                                               _stream_handle(stream))
    _check(st, "decode_gemm_bf16_reduce_rmsnorm")
    return out, residual_out


def gather_shards_bf16(shards, out, stream=None):
    """out[M, TP*S] = the TP shards [TP, M, S] side by side (rank r at columns r*S..).

    shards, out: contiguous CUDA bfloat16 tensors. Returns ``out``.
    """
    _bf16_cuda(shards, "shards")
    if shards.dim() != 3:
        raise ValueError(f"shards must be [TP, M, S], got {tuple(shards.shape)}")
    TP, M, S = shards.shape
    _bf16_cuda(out, "out", (M, TP * S))
    st = load_library().gather_shards_bf16(shards.data_ptr(), TP, M, S, out.data_ptr(),
                                           _stream_handle(stream))
    _check(st, "gather_shards_bf16")
    return out


def _type_error(t, name, dtype):
    """The exception for a t that is no CUDA tensor of a dtype."""
    if not (hasattr(t, "dtype") and hasattr(t, "device")):
        return TypeError(f"{name} must be a torch.Tensor")
    return TypeError(f"{name} must be a CUDA {dtype} tensor (got {t.dtype} on {t.device})")


def _rows(t, name, bf16, width=None, rows=None):
    """A CUDA bfloat16 tensor whose rows (all but its first axis) are contiguous: the
    stride between rows, in elements (the row's width for a single row)."""
    try:
        good = t.dtype == bf16 and t.is_cuda
    except AttributeError:
        good = False
    if not good:
        raise _type_error(t, name, bf16)
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must have rows")
    if rows is not None and shape[0] != rows:
        raise ValueError(f"{name} has {shape[0]} rows, expected {rows}")
    stride = t.stride()
    n = 1
    for i in range(len(shape) - 1, 0, -1):
        if stride[i] != n and shape[i] != 1:
            raise ValueError(f"{name}'s rows must be contiguous")
        n *= shape[i]
    if width is not None and n != width:
        raise ValueError(f"{name} has rows of {n}, expected {width}")
    return stride[0] if shape[0] > 1 else n


def _plain_cuda(t, name, dtype, shape):
    """The address of a contiguous CUDA tensor of a dtype and shape."""
    try:
        good = t.dtype == dtype and t.is_cuda
    except AttributeError:
        good = False
    if not good:
        raise _type_error(t, name, dtype)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _cache_fields(k_cache, v_cache, bf16):
    """The fields of skinny_kv_cache for two [pages, page_size, kv_heads, head_dim] views."""
    bad = (k_cache, "k_cache")
    try:
        good = k_cache.dtype == bf16 and k_cache.is_cuda
        if good:
            bad = (v_cache, "v_cache")
            good = v_cache.dtype == bf16 and v_cache.is_cuda
    except AttributeError:
        good = False
    if not good:
        raise _type_error(*bad, bf16)
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache {tuple(shape)} and v_cache {tuple(v_cache.shape)} must be "
                         "[pages, page_size, kv_heads, head_dim]")
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks != vs or ks[3] != 1 or (ks[0] | ks[1] | ks[2]) & 7:
        # The stride of an axis of one element says nothing.
        ks, vs = ([0 if n == 1 else st for n, st in zip(shape, t)] for t in (ks, vs))
        if ks != vs or (ks[3] != 1 and shape[3] != 1):
            raise ValueError("k_cache and v_cache must have the same strides, 1 along head_dim")
    return k_cache.data_ptr(), v_cache.data_ptr(), *shape, ks[0], ks[1], ks[2]


def qk_norm_rope_bf16(qkv, q_heads, kv_heads, q_gamma, k_gamma, rope, positions, q_out, k_out=None,
                      k_cache=None, v_cache=None, slots=None, eps=1e-6, interleaved=False,
                      stream=None, pdl=None):
    """Per-head RMSNorm and position rotation of QKV rows, and the append to a paged cache.

    qkv [M, (q_heads + 2 kv_heads) * head_dim], rows contiguous, any row stride;
    q_gamma, k_gamma [head_dim] or None (no norm); rope [max_pos, rot_dim] FP32
    (cosines, then sines) or None (no rotation); positions [M] int32. q_out [M, q_heads,
    head_dim] (or flat rows; may be qkv's own query heads, in place); k_out [M, kv_heads,
    head_dim] or None. k_cache, v_cache: [pages, page_size, kv_heads, head_dim] views of
    equal strides, or None; slots [M] int64 (page * page_size + token; negative: not
    stored). Returns ``q_out``.
    """
    import torch
    bf16 = torch.bfloat16
    qkv_stride = _rows(qkv, "qkv", bf16)
    shape = qkv.shape
    heads = q_heads + 2 * kv_heads
    if len(shape) != 2 or q_heads < 1 or kv_heads < 1 or shape[1] % heads:
        raise ValueError(f"qkv {tuple(shape)} must be [M, ({q_heads} + 2 * {kv_heads}) * head_dim]")
    M = shape[0]
    D = shape[1] // heads
    q_stride = _rows(q_out, "q_out", bf16, q_heads * D, M)
    k_ptr = k_stride = q_gamma_ptr = k_gamma_ptr = rope_ptr = positions_ptr = slots_ptr = 0
    max_pos = rot_dim = 0
    cache = _NO_CACHE
    if k_out is not None:
        k_stride, k_ptr = _rows(k_out, "k_out", bf16, kv_heads * D, M), k_out.data_ptr()
    if q_gamma is not None:
        q_gamma_ptr = _plain_cuda(q_gamma, "q_gamma", bf16, (D,))
    if k_gamma is not None:
        k_gamma_ptr = _plain_cuda(k_gamma, "k_gamma", bf16, (D,))
    if rope is not None:
        shape = getattr(rope, "shape", None)
        rope_ptr = _plain_cuda(rope, "rope", torch.float32, shape)
        if len(shape) != 2:
            raise ValueError(f"rope must be [max_pos, rot_dim], got {tuple(shape)}")
        max_pos, rot_dim = shape
        positions_ptr = _plain_cuda(positions, "positions", torch.int32, (M,))
    if k_cache is not None or v_cache is not None:
        if k_cache is None or v_cache is None or slots is None:
            raise ValueError("k_cache, v_cache and slots go together")
        cache = _cache_fields(k_cache, v_cache, bf16)
        slots_ptr = _plain_cuda(slots, "slots", torch.int64, (M,))
    try:
        a = _pack_rope(qkv.data_ptr(), qkv_stride, M, q_heads, kv_heads, D, q_gamma_ptr, k_gamma_ptr, eps,
                       rope_ptr, max_pos, rot_dim, bool(interleaved), positions_ptr, q_out.data_ptr(), q_stride,
                       k_ptr, k_stride, *cache, slots_ptr)
    except struct.error as e:  # a number of the wrong kind, or past the field's range
        raise ValueError(f"qk_norm_rope_bf16: {e}") from None
    o = _opts(pdl, None)
    st = load_library().qk_norm_rope_bf16(a, None if o is None else ctypes.byref(o),
                                          _stream_handle(stream))
    _check(st, "qk_norm_rope_bf16")
    return q_out


ATTENTION_COUNTER_BYTES = 8192


def attention_workspace(device=None):
    """A workspace for decode_attention_bf16 on a device, made ready on the current stream;
    every call leaves it ready for the next. Calls that may run at the same time need one
    each."""
    import torch
    dev = torch.cuda.current_device() if device is None else device
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    ws = torch.empty(load_library().skinny_attention_workspace_bytes(sms), dtype=torch.uint8,
                     device=torch.device("cuda", dev) if isinstance(dev, int) else dev)
    ws[:ATTENTION_COUNTER_BYTES].zero_()
    return ws


_workspaces = {}  # (device, stream) -> the workspace of calls that bring none


def _own_workspace(device, stream, find=None, *args):
    """The workspace of a call on ``stream`` (a handle) that brings none. Calls on one
    stream run one after another and share one; a call being captured gets its own,
    zeroed in the graph, so that graphs replayed side by side do not meet. Both are made
    with the launch stream current, whatever the caller's is: the zeroing comes before
    the kernel, and the memory goes to no other stream's call while the kernel runs."""
    import torch
    find = find or _current_workspace
    handle = stream.value or 0
    if handle != torch._C._cuda_getCurrentRawStream(device):
        on = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
        with torch.cuda.stream(on):
            return find(device, handle, *args)
    return find(device, handle, *args)


def _current_workspace(device, handle):
    import torch
    if torch._C._cuda_isCurrentStreamCapturing():
        return attention_workspace(device)
    ws = _workspaces.get((device, handle))
    if ws is None:
        ws = _workspaces.setdefault((device, handle), attention_workspace(device))
    return ws


def decode_attention_bf16(q, k_cache, v_cache, block_table, lengths, out, scale=None, window=0,
                          sinks=0, lse=None, workspace=None, stream=None, pdl=None):
    """Attention of one new token per row over a paged key-value cache.

    q [rows, q_heads, head_dim], each row contiguous, any row stride; k_cache, v_cache
    [pages, page_size, kv_heads, head_dim] views of equal strides; block_table [rows,
    table_width] int32; lengths [rows] int32; out like q, contiguous; lse [rows, q_heads]
    FP32 or None. scale: 1 / sqrt(head_dim) if None. window > 0: a row sees its last
    ``window`` tokens and its first ``sinks``. workspace: attention_workspace(), or None
    for one kept per stream; a call whose stream is captured by torch.cuda.graph gets its
    own (a capture begun by other means needs a workspace that lives as long as its graph).
    Returns ``out``.
    """
    import torch
    bf16 = torch.bfloat16
    q_stride = _rows(q, "q", bf16)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError(f"q must be [rows, q_heads, head_dim], got {tuple(shape)}")
    rows, q_heads, D = shape
    cache = _cache_fields(k_cache, v_cache, bf16)
    if cache[5] != D:
        raise ValueError(f"q has heads of {D}, the cache of {cache[5]}")
    out_ptr = _plain_cuda(out, "out", bf16, shape)
    try:
        good = block_table.dtype == torch.int32 and block_table.is_cuda
    except AttributeError:
        good = False
    if not good:
        raise _type_error(block_table, "block_table", torch.int32)
    table_shape, table_stride = block_table.shape, block_table.stride()
    if len(table_shape) != 2 or table_shape[0] != rows or (table_stride[1] != 1 and table_shape[1] > 1):
        raise ValueError(f"block_table must be [{rows}, table_width] with contiguous rows")
    lengths_ptr = _plain_cuda(lengths, "lengths", torch.int32, (rows,))
    lse_ptr = 0 if lse is None else _plain_cuda(lse, "lse", torch.float32, (rows, q_heads))
    handle = _stream_handle(stream)
    if workspace is None:
        device = q.device.index
        if stream is None:
            workspace = _current_workspace(device, handle.value or 0)
        elif device != torch._C._cuda_getDevice():
            _check(4, "decode_attention_bf16")  # as the call itself would say
        else:
            workspace = _own_workspace(device, handle)
    elif not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    width = table_shape[1]
    try:
        a = _pack_attention(
            q.data_ptr(), q_stride, rows, q_heads, *cache, block_table.data_ptr(),
            table_stride[0] if rows > 1 else width, width, lengths_ptr, window, sinks,
            D ** -0.5 if scale is None else scale, out_ptr, lse_ptr, workspace.data_ptr(), workspace.nbytes)
    except struct.error as e:  # a number of the wrong kind, or past the field's range
        raise ValueError(f"decode_attention_bf16: {e}") from None
    o = _opts(pdl, None)
    st = load_library().decode_attention_bf16(a, None if o is None else ctypes.byref(o), handle)
    _check(st, "decode_attention_bf16")
    return out


def token_logprobs_bf16(logits, tokens, logprobs, entropy=None, lse=None, top_logprobs=None,
                        top_tokens=None, stream=None, pdl=None):
    """Log probabilities of given tokens, the entropy and the most likely tokens of rows of logits.

    logits [M, V] bfloat16, rows contiguous, any row stride; tokens [M] or [M, given] int64
    (negative: not asked for, 0 comes out) or None; logprobs FP32 of tokens' shape (None if
    tokens is); entropy, lse [M] FP32 or None; top_logprobs [M, top] FP32 and top_tokens
    [M, top] int64, either or both None; top <= min(V, 32), of equal logits the lower index
    first. Returns ``logprobs``.
    """
    import torch
    stride = _rows(logits, "logits", torch.bfloat16)
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError(f"logits must be [M, V], got {tuple(shape)}")
    M, V = shape
    f32, i64 = torch.float32, torch.int64
    given = top = tokens_ptr = logprobs_ptr = entropy_ptr = lse_ptr = top_lp_ptr = top_tok_ptr = 0
    if tokens is not None or logprobs is not None:
        if tokens is None or logprobs is None:
            raise ValueError("tokens and logprobs go together")
        shape = getattr(tokens, "shape", ())
        tokens_ptr = _plain_cuda(tokens, "tokens", i64, shape)
        if len(shape) not in (1, 2) or shape[0] != M:
            raise ValueError(f"tokens must be [{M}] or [{M}, given], got {tuple(shape)}")
        given = shape[1] if len(shape) == 2 else 1
        logprobs_ptr = _plain_cuda(logprobs, "logprobs", f32, shape)
    if entropy is not None:
        entropy_ptr = _plain_cuda(entropy, "entropy", f32, (M,))
    if lse is not None:
        lse_ptr = _plain_cuda(lse, "lse", f32, (M,))
    if top_logprobs is not None or top_tokens is not None:
        shape = getattr(top_tokens if top_logprobs is None else top_logprobs, "shape", ())
        if len(shape) != 2 or shape[0] != M:
            raise ValueError(f"top_logprobs and top_tokens must be [{M}, top]")
        top = shape[1]
        if top_logprobs is not None:
            top_lp_ptr = _plain_cuda(top_logprobs, "top_logprobs", f32, shape)
        if top_tokens is not None:
            top_tok_ptr = _plain_cuda(top_tokens, "top_tokens", i64, shape)
    try:
        a = _pack_logprobs(logits.data_ptr(), stride, M, V, tokens_ptr, given, logprobs_ptr, entropy_ptr, lse_ptr,
                           top, top_lp_ptr, top_tok_ptr)
    except struct.error as e:  # a size past the field's range
        raise ValueError(f"token_logprobs_bf16: {e}") from None
    o = _opts(pdl, None)
    st = load_library().token_logprobs_bf16(a, None if o is None else ctypes.byref(o), _stream_handle(stream))
    _check(st, "token_logprobs_bf16")
    return logprobs


def shared_prefix_workspace(rows, q_heads, kv_heads, head_dim, device=None):
    """A workspace for decode_attention_shared_prefix_bf16 of up to these rows and query heads
    on a device, made ready on the current stream; every call leaves it ready for the next.
    Calls that may run at the same time need one each."""
    import torch
    dev = torch.cuda.current_device() if device is None else device
    n = _prefix_bytes(rows, q_heads, kv_heads, head_dim, dev)
    if not n:
        raise ValueError(f"no shared-prefix attention of {rows} rows, {q_heads} heads on {kv_heads}, {head_dim} wide")
    return _zeroed(n, dev)


_sms = {}  # device -> its SMs


def _prefix_bytes(rows, q_heads, kv_heads, head_dim, dev):
    import torch
    sms = _sms.get(dev)
    if sms is None:
        sms = _sms[dev] = torch.cuda.get_device_properties(dev).multi_processor_count
    return load_library().skinny_shared_prefix_workspace_bytes(rows, q_heads, kv_heads, head_dim, sms)


def _zeroed(n, dev):
    """n bytes on a device, the counters at their start zero."""
    import torch
    ws = torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", dev) if isinstance(dev, int) else dev)
    ws[:ATTENTION_COUNTER_BYTES].zero_()
    return ws


_prefix_workspaces = {}  # (device, stream) -> the workspace of calls that bring none


def _current_prefix_workspace(device, handle, n):
    """As _current_workspace, of n bytes or more: a larger one takes a smaller one's place,
    whose memory the stream's next allocations get behind the calls that use it."""
    import torch
    if torch._C._cuda_isCurrentStreamCapturing():
        return _zeroed(n, device)
    ws = _prefix_workspaces.get((device, handle))
    if ws is None or ws.nbytes < n:
        ws = _prefix_workspaces[(device, handle)] = _zeroed(n, device)
    return ws


def decode_attention_shared_prefix_bf16(q, k_cache, v_cache, prefix_table, prefix_length, block_table, lengths,
                                        out, scale=None, lse=None, workspace=None, stream=None, pdl=None):
    """Attention of one new token per row over a prefix that all rows share and the row's own
    tokens after it, both in a paged key-value cache; the prefix is read once for all rows.

    prefix_table [prefix_width] int32: the prefix's pages; prefix_length [1] int32 on the
    device. block_table [rows, table_width] and lengths [rows] int32 are of the rows' own
    tokens (a row of length 0 sees the prefix alone). workspace: shared_prefix_workspace(), or
    None for one kept per stream, as in decode_attention_bf16, which the other arguments
    follow too. Returns ``out``.
    """
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    q_stride = _rows(q, "q", bf16)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError(f"q must be [rows, q_heads, head_dim], got {tuple(shape)}")
    rows, q_heads, D = shape
    cache = _cache_fields(k_cache, v_cache, bf16)
    if cache[5] != D:
        raise ValueError(f"q has heads of {D}, the cache of {cache[5]}")
    out_ptr = _plain_cuda(out, "out", bf16, shape)
    prefix_shape = getattr(prefix_table, "shape", ())
    prefix_ptr = _plain_cuda(prefix_table, "prefix_table", i32, prefix_shape)
    if len(prefix_shape) != 1:
        raise ValueError(f"prefix_table must be [prefix_width], got {tuple(prefix_shape)}")
    length_ptr = _plain_cuda(prefix_length, "prefix_length", i32, (1,))
    try:
        good = block_table.dtype == i32 and block_table.is_cuda
    except AttributeError:
        good = False
    if not good:
        raise _type_error(block_table, "block_table", i32)
    table_shape, table_stride = block_table.shape, block_table.stride()
    if len(table_shape) != 2 or table_shape[0] != rows or (table_stride[1] != 1 and table_shape[1] > 1):
        raise ValueError(f"block_table must be [{rows}, table_width] with contiguous rows")
    lengths_ptr = _plain_cuda(lengths, "lengths", i32, (rows,))
    lse_ptr = 0 if lse is None else _plain_cuda(lse, "lse", torch.float32, (rows, q_heads))
    handle = _stream_handle(stream)
    if workspace is None:
        device = q.device.index
        if device != torch._C._cuda_getDevice():
            _check(4, "decode_attention_shared_prefix_bf16")  # as the call itself would say
        n = _prefix_bytes(rows, q_heads, cache[4], D, device)
        if not n:
            _check(2, "decode_attention_shared_prefix_bf16")
        workspace = _own_workspace(device, handle, _current_prefix_workspace, n)
    elif not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    width = table_shape[1]
    try:
        a = _pack_prefix(
            q.data_ptr(), q_stride, rows, q_heads, *cache, prefix_ptr, prefix_shape[0], length_ptr,
            block_table.data_ptr(), table_stride[0] if rows > 1 else width, width, lengths_ptr,
            D ** -0.5 if scale is None else scale, out_ptr, lse_ptr, workspace.data_ptr(), workspace.nbytes)
    except struct.error as e:  # a number of the wrong kind, or past the field's range
        raise ValueError(f"decode_attention_shared_prefix_bf16: {e}") from None
    o = _opts(pdl, None)
    st = load_library().decode_attention_shared_prefix_bf16(a, None if o is None else ctypes.byref(o), handle)
    _check(st, "decode_attention_shared_prefix_bf16")
    return out


def device_error(device=None):
    """(status, word): read and clear the library's device error word."""
    import torch
    dev = torch.cuda.current_device() if device is None else int(device)
    word = ctypes.c_int(0)
    st = load_library().skinny_device_error(dev, ctypes.byref(word))
    return st, word.value


def set_pdl(enable: bool) -> bool:
    """Enable or disable programmatic dependent launch; returns the old setting."""
    return bool(load_library().skinny_set_pdl(1 if enable else 0))


def set_l2_prefetch(blocks: int) -> int:
    """Weight blocks the decode GEMM's deep ring prefetches to L2 before its PDL
    wait (skinny_set_l2_prefetch); returns the old value."""
    prev = load_library().skinny_set_l2_prefetch(int(blocks))
    if prev < 0:
        raise ValueError(f"l2 prefetch blocks must be in [0, 64], got {blocks}")
    return prev


def gemm_plan(M, N, K, num_sms) -> GemmPlan:
    plan = GemmPlan()
    _check(load_library().skinny_gemm_plan_query(M, N, K, num_sms, ctypes.byref(plan)),
           "skinny_gemm_plan_query")
    return plan


def gemm_cta_pieces(M, N, K, num_sms, cta, max_pieces=64):
    """[(tile, kb0, kb1, slot)] of one CTA of the decode GEMM's work split."""
    arrs = [(ctypes.c_int * max_pieces)() for _ in range(4)]
    n = load_library().skinny_gemm_cta_pieces(M, N, K, num_sms, cta, *arrs, max_pieces)
    if n < 0:
        raise ValueError("bad arguments to skinny_gemm_cta_pieces")
    return [tuple(a[i] for a in arrs) for i in range(min(n, max_pieces))]


def watchdog_selftest(x, W, out, timeout_ns, stream=None):
    """Launch the decode GEMM with a wait that can never complete (see skinny.h)."""
    M, K = x.shape
    N = W.shape[0]
    st = load_library().skinny_watchdog_selftest(x.data_ptr(), W.data_ptr(), out.data_ptr(),
                                                 M, N, K, int(timeout_ns),
                                                 _stream_handle(stream))
    _check(st, "skinny_watchdog_selftest")


def reduce_selftest(partials, residual, gamma, out, residual_out, eps, timeout_ns, stream=None):
    """Launch the reduce with a cluster exchange that can never complete (see skinny.h)."""
    _bf16_cuda(partials, "partials")
    if partials.dim() != 3 or partials.shape[2] != HIDDEN:
        raise ValueError(f"partials must be [TP, M, {HIDDEN}], got {tuple(partials.shape)}")
    TP, M, _ = partials.shape
    if residual is not None:
        _bf16_cuda(residual, "residual", (M, HIDDEN))
    _bf16_cuda(gamma, "gamma", (HIDDEN,))
    _bf16_cuda(out, "out", (M, HIDDEN))
    _bf16_cuda(residual_out, "residual_out", (M, HIDDEN))
    st = load_library().skinny_reduce_selftest(
        partials.data_ptr(), TP, residual.data_ptr() if residual is not None else None,
        gamma.data_ptr(), out.data_ptr(), residual_out.data_ptr(), M, float(eps),
        int(timeout_ns), _stream_handle(stream))
    _check(st, "skinny_reduce_selftest")


def shared_prefix_selftest(q, k_cache, v_cache, prefix_table, prefix_length, block_table, lengths, out, lse,
                           workspace, timeout_ns, stream=None):
    """Launch the shared-prefix attention with a wait that can never complete (see skinny.h)."""
    import torch
    rows, q_heads, D = q.shape
    st = load_library().skinny_shared_prefix_selftest(
        _pack_prefix(q.data_ptr(), _rows(q, "q", torch.bfloat16), rows, q_heads,
                     *_cache_fields(k_cache, v_cache, torch.bfloat16), prefix_table.data_ptr(),
                     prefix_table.numel(), prefix_length.data_ptr(), block_table.data_ptr(),
                     block_table.stride(0), block_table.shape[1], lengths.data_ptr(), D ** -0.5,
                     out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes),
        int(timeout_ns), _stream_handle(stream))
    _check(st, "skinny_shared_prefix_selftest")
