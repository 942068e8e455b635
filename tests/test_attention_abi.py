"""Refusals of the decode attention, the per-head norm with rotation and the GEMM epilogue
without a GPU: every bad argument is reported before anything touches CUDA."""
import ctypes

import pytest

import skinny_bf16_gemm_gb300 as sk
from skinny_bf16_gemm_gb300 import build as skbuild

NULL, SHAPE, ALIGN, DEVICE, ALIAS, ARG = 1, 2, 3, 4, 6, 10


@pytest.fixture(scope="module")
def lib():
    skbuild.build()
    return sk.load_library()


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(32 << 20)
    return buf, ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 4096


MB = 1 << 20


def cache_at(p, **kw):
    c = dict(k=p, v=p + MB, num_pages=4, page_size=16, kv_heads=2, head_dim=64,
             page_stride=16 * 128, token_stride=128, head_stride=64)
    c.update(kw)
    return sk.KVCacheArgs(**c)


def test_epilogue_refusals(lib, mem):
    _, p = mem
    f = lib.decode_gemm_bf16_epilogue
    names = ["x", "W", "bias", "res", "out", "M", "N", "K", "act", "opts", "s"]
    ok = dict(zip(names, (p, p + MB, p + 2 * MB, p + 3 * MB, p + 4 * MB, 4, 16, 64, 2, None, None)))

    def call(**kw):
        return f(*[dict(ok, **kw)[n] for n in names])
    for n in ("x", "W", "out"):
        assert call(**{n: None}) == NULL
    assert call(act=-1) == ARG and call(act=5) == ARG
    assert call(M=0) == SHAPE and call(M=65) == SHAPE and call(K=12) == SHAPE and call(N=0) == SHAPE
    assert call(x=p + 8) == ALIGN and call(bias=p + 2 * MB + 1) == ALIGN
    assert call(res=p + 3 * MB + 1) == ALIGN and call(out=p + 4 * MB + 1) == ALIGN
    assert call(out=p + 64) == ALIAS and call(out=p + MB + 64) == ALIAS
    assert call(out=p + 2 * MB) == ALIAS            # over the bias
    assert call(out=p + 3 * MB + 2) == ALIAS        # residual, shifted
    bad = ctypes.byref(sk.LaunchOpts(2, 0))
    assert call(opts=bad) == ARG
    import torch
    if not torch.cuda.is_available():
        for kw in ({}, {"out": p + 3 * MB}, {"bias": None}, {"res": None}, {"bias": None, "res": None}):
            assert call(**kw) == DEVICE              # valid (in place too), but no device
    with pytest.raises(TypeError):
        sk.decode_gemm_bf16_epilogue(torch.zeros(1, 8), torch.zeros(8, 8), torch.zeros(1, 8))


def rope_args(p, cache=None, **kw):
    a = dict(qkv=p, qkv_stride=8 * 64, M=3, q_heads=4, kv_heads=2, head_dim=64, q_gamma=p + 2 * MB,
             k_gamma=p + 2 * MB + 4096, eps=1e-6, rope=p + 3 * MB, max_pos=32, rot_dim=64,
             interleaved=0, positions=p + 4 * MB, q_out=p + 5 * MB, q_stride=4 * 64,
             k_out=p + 6 * MB, k_stride=2 * 64, slots=p + 7 * MB)
    a.update(kw)
    args = sk.QkNormRopeArgs(**a)
    if cache is not None:
        args.cache = cache
    return args


def test_qk_norm_rope_refusals(lib, mem):
    _, p = mem

    def call(cache=None, opts=None, **kw):
        a = rope_args(p, cache, **kw)
        return lib.qk_norm_rope_bf16(ctypes.byref(a), opts, None)
    assert lib.qk_norm_rope_bf16(None, None, None) == NULL
    for n in ("qkv", "q_out", "rope", "positions"):
        assert call(**{n: None}) == NULL
    good = cache_at(p + 8 * MB)
    assert call(cache=good, slots=None) == NULL
    assert call(cache=cache_at(p, k=None)) == NULL
    for kw in (dict(M=0), dict(q_heads=0), dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=60),
               dict(head_dim=0), dict(head_dim=264), dict(rot_dim=24), dict(rot_dim=80),
               dict(rot_dim=-16), dict(max_pos=0), dict(qkv_stride=8 * 64 - 8),
               dict(q_stride=4 * 64 - 8), dict(k_stride=64)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(interleaved=2)):
        assert call(**kw) == ARG, kw
    for kw in (dict(qkv=p + 8), dict(q_out=p + 5 * MB + 8), dict(k_out=p + 6 * MB + 8),
               dict(rope=p + 3 * MB + 4), dict(positions=p + 4 * MB + 2), dict(q_gamma=p + 2 * MB + 2),
               dict(slots=p + 7 * MB + 4), dict(qkv_stride=8 * 64 + 4)):
        assert call(cache=good, **kw) == ALIGN, kw
    for kw in (dict(q_out=p), dict(q_out=p + 256, q_stride=512), dict(k_out=p, k_stride=512),
               dict(k_out=p + 5 * MB), dict(q_out=p + 3 * MB), dict(q_out=p + 4 * MB),
               dict(q_out=p + 2 * MB), dict(q_out=p + 7 * MB), dict(q_out=p + 8 * MB + 4096)):
        assert call(cache=good, **kw) == ALIAS, kw
    for bad, code in ((dict(num_pages=0), SHAPE), (dict(page_size=0), SHAPE), (dict(kv_heads=1), SHAPE),
                      (dict(head_dim=128), SHAPE), (dict(token_stride=-8), SHAPE),
                      (dict(page_stride=1 << 41), SHAPE), (dict(token_stride=132), ALIGN),
                      (dict(k=p + 8 * MB + 8), ALIGN), (dict(token_stride=0), ALIAS),
                      (dict(head_stride=32), ALIAS), (dict(v=p + 8 * MB), ALIAS)):
        assert call(cache=cache_at(p + 8 * MB, **bad)) == code, bad
    assert call(opts=ctypes.byref(sk.LaunchOpts(-2, 0))) == ARG
    import torch
    if not torch.cuda.is_available():
        for kw in ({}, dict(q_out=p, q_stride=512), dict(k_out=p + 512, k_stride=512), dict(k_out=None),
                   dict(q_out=p, q_stride=512, k_out=p + 512, k_stride=512),
                   dict(rot_dim=0, rope=None, positions=None), dict(q_gamma=None, k_gamma=None)):
            assert call(cache=good, **kw) == DEVICE, kw


def test_decode_attention_refusals(lib, mem):
    _, p = mem
    size = sk.load_library().skinny_attention_workspace_bytes(152)
    assert lib.skinny_attention_workspace_bytes(0) == 0 and size > 0 and size % 16 == 0
    ok = dict(q=p, q_stride=256, rows=3, q_heads=4, block_table=p + 2 * MB, table_stride=4, table_width=4,
              lengths=p + 3 * MB, window=0, sinks=0, scale=0.125, out=p + 4 * MB, lse=p + 5 * MB,
              workspace=p + 8 * MB, workspace_bytes=size)

    def call(cache=None, opts=None, **kw):
        a = sk.DecodeAttentionArgs(**dict(ok, **kw))
        a.cache = cache if cache is not None else cache_at(p + 6 * MB, v=p + 7 * MB)
        return lib.decode_attention_bf16(ctypes.byref(a), opts, None)
    assert lib.decode_attention_bf16(None, None, None) == NULL
    assert call(cache=cache_at(p, k=None)) == NULL and call(cache=cache_at(p, v=None)) == NULL
    for n in ("q", "block_table", "lengths", "out", "workspace"):
        assert call(**{n: None}) == NULL, n
    for kw in (dict(rows=0), dict(rows=1025), dict(q_heads=3), dict(q_heads=0), dict(q_heads=1026),
               dict(table_width=0), dict(table_stride=3), dict(q_stride=248),
               dict(table_width=1 << 26, table_stride=1 << 26)):
        assert call(**kw) == SHAPE, kw
    for D in (8, 72, 120, 136, 248):
        assert call(cache=cache_at(p + 6 * MB, head_dim=D)) == SHAPE
    for kw in (dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**kw) == ARG, kw
    for kw in (dict(q=p + 8), dict(out=p + 4 * MB + 8), dict(workspace=p + 8 * MB + 8),
               dict(block_table=p + 2 * MB + 2), dict(lengths=p + 3 * MB + 2), dict(lse=p + 5 * MB + 2),
               dict(q_stride=260)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(out=p), dict(out=p + 2 * MB), dict(out=p + 3 * MB), dict(out=p + 6 * MB),
               dict(out=p + 7 * MB + 256), dict(lse=p), dict(lse=p + 4 * MB), dict(workspace=p + 7 * MB),
               dict(out=p + 8 * MB + 4096)):
        assert call(**kw) == ALIAS, kw
    assert call(opts=ctypes.byref(sk.LaunchOpts(2, 0))) == ARG
    import torch
    if not torch.cuda.is_available():
        for kw in ({}, dict(lse=None), dict(window=5, sinks=2), dict(scale=-1.0)):
            assert call(**kw) == DEVICE, kw


def test_table_too_wide_for_32_bit_tiles_is_refused(lib, mem):
    """1024 rows x 1024 heads x tables of 2^24 tokens: more than 2^31 tiles."""
    _, p = mem
    c = cache_at(p + 6 * MB, v=p + 7 * MB, kv_heads=1024, head_stride=0, token_stride=0, page_stride=0)
    a = sk.DecodeAttentionArgs(q=p, q_stride=65536, rows=1024, q_heads=1024, block_table=p, table_stride=1 << 20,
                               table_width=1 << 20, lengths=p, scale=1.0, out=p, workspace=p,
                               workspace_bytes=1 << 30)
    a.cache = c
    assert lib.decode_attention_bf16(ctypes.byref(a), None, None) == SHAPE


def test_python_checks_name_the_tensor(lib):
    import torch
    t = torch.zeros(4, 8 * 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="qkv"):
        sk.qk_norm_rope_bf16(t, 4, 2, None, None, None, None, t)
    with pytest.raises(TypeError, match="q must be"):
        sk.decode_attention_bf16(t.view(4, 8, 64), t, t, None, None, None)
    with pytest.raises(ValueError, match="activation"):
        class Fake(torch.Tensor):
            is_cuda = True
        x = torch.zeros(1, 8, dtype=torch.bfloat16).as_subclass(Fake)
        sk.decode_gemm_bf16_epilogue(x, x, torch.zeros(1, 1, dtype=torch.bfloat16).as_subclass(Fake),
                                     activation="tanh")


def test_packed_strings_match_the_structures(lib):
    """The wrappers fill the two argument structures as packed strings: the same bytes."""
    n = iter(range(1, 100))
    cache = [next(n) for _ in range(9)]
    rope = [next(n) for _ in range(18)]
    packed = sk._pack_rope(*rope, *cache, 98)
    a = sk.QkNormRopeArgs(*rope, sk.KVCacheArgs(*cache), 98)
    assert bytes(a) == packed
    first, last = [next(n) for _ in range(4)], [next(n) for _ in range(11)]
    assert bytes(sk.DecodeAttentionArgs(*first, sk.KVCacheArgs(*cache), *last)) == \
        sk._pack_attention(*first, *cache, *last)


def test_new_status_has_a_text(lib):
    assert sk.status_string(11) != "unknown status" and sk.STATUS[11] == "SKINNY_ERR_INDEX"
