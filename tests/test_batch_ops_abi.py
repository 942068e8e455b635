"""Refusals of the adapters' linear, the shared-prefix attention and the log probabilities
without a GPU: every bad argument is reported before anything touches CUDA, in the C calls
and in the wrappers; and the plan of the shared prefix, checked by itself."""
import ctypes

import pytest

import skinny_bf16_gemm_gb300 as sk
from test_attention_abi import ALIAS, ALIGN, ARG, DEVICE, MB, NULL, SHAPE, cache_at, lib, mem  # noqa: F401
from test_decoder_ops_refusals import fake_cuda


def no_device():
    import torch
    return not torch.cuda.is_available()


def logprob_args(p, **kw):
    a = dict(logits=p, logits_stride=1008, M=3, V=1001, tokens=p + MB, given=2, logprobs=p + 2 * MB,
             entropy=p + 3 * MB, lse=p + 4 * MB, top=5, top_logprobs=p + 5 * MB, top_tokens=p + 6 * MB)
    a.update(kw)
    return sk.TokenLogprobsArgs(**a)


def test_token_logprobs_refusals(lib, mem):
    _, p = mem

    def call(opts=None, **kw):
        return lib.token_logprobs_bf16(bytes(logprob_args(p, **kw)), opts, None)
    assert lib.token_logprobs_bf16(None, None, None) == NULL
    for n in ("logits", "tokens", "logprobs"):
        assert call(**{n: None}) == NULL, n
    assert call(given=0, entropy=None, lse=None, top=0) == NULL                  # nothing asked for
    assert call(given=0, entropy=None, lse=None, top_logprobs=None, top_tokens=None) == NULL
    for kw in (dict(M=0), dict(M=(1 << 24) + 1), dict(V=0), dict(V=(1 << 30) + 1), dict(given=-1),
               dict(given=(1 << 20) + 1), dict(top=-1), dict(top=33), dict(V=4, logits_stride=8),
               dict(logits_stride=1000), dict(logits_stride=(1 << 32) + 1)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(logits=p + 1), dict(tokens=p + MB + 4), dict(logprobs=p + 2 * MB + 2),
               dict(entropy=p + 3 * MB + 2), dict(lse=p + 4 * MB + 2), dict(top_logprobs=p + 5 * MB + 2),
               dict(top_tokens=p + 6 * MB + 4)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(logprobs=p + 4000), dict(entropy=p + MB + 40), dict(lse=p), dict(top_logprobs=p + MB),
               dict(top_tokens=p + 16), dict(lse=p + 3 * MB + 8), dict(top_logprobs=p + 2 * MB + 20),
               dict(top_tokens=p + 5 * MB + 56)):
        assert call(**kw) == ALIAS, kw
    assert call(opts=ctypes.byref(sk.LaunchOpts(2, 0))) == ARG
    if no_device():
        for kw in ({}, dict(logits=p + 2), dict(given=0, tokens=None, logprobs=None), dict(entropy=None, lse=None),
                   dict(top=0, top_logprobs=None, top_tokens=None), dict(top_logprobs=None), dict(top=0),
                   dict(top_tokens=None), dict(V=32, top=32), dict(M=1, logits_stride=1001)):
            assert call(**kw) == DEVICE, kw


def test_lora_refusals(lib, mem):
    _, p = mem
    names = ["x", "W", "lora", "bias", "res", "out", "M", "N", "K", "act", "opts", "s"]
    ok = dict(zip(names, (p, p + MB, None, p + 2 * MB, p + 3 * MB, p + 4 * MB, 4, 16, 64, 2, None, None)))

    def call(lora=True, A=p + 5 * MB, B=p + 6 * MB, adapters=p + 7 * MB, scales=p + 8 * MB, num_adapters=3, rank=16, **kw):
        a = bytes(sk.LoraArgs(A, B, adapters, scales, num_adapters, rank)) if lora else None
        return lib.decode_gemm_bf16_lora(*[dict(ok, lora=a, **kw)[n] for n in names])
    assert call(lora=False) == NULL
    for n in ("x", "W", "out", "A", "B", "adapters"):
        assert call(**{n: None}) == NULL, n
    for kw in (dict(rank=0), dict(rank=4), dict(rank=12), dict(rank=136), dict(rank=-8), dict(num_adapters=0),
               dict(num_adapters=(1 << 20) + 1), dict(M=0), dict(M=65), dict(K=12), dict(N=0)):
        assert call(**kw) == SHAPE, kw
    assert call(act=5) == ARG and call(act=-1) == ARG
    for kw in (dict(A=p + 5 * MB + 8), dict(B=p + 6 * MB + 8), dict(adapters=p + 7 * MB + 2),
               dict(scales=p + 8 * MB + 2), dict(x=p + 8), dict(bias=p + 2 * MB + 1), dict(out=p + 4 * MB + 1)):
        assert call(**kw) == ALIGN, kw
    for out in (p, p + MB, p + 2 * MB, p + 3 * MB + 2, p + 5 * MB, p + 6 * MB + 64, p + 7 * MB + 8, p + 8 * MB + 4):
        assert call(out=out) == ALIAS, (out - p) / MB
    assert call(out=p + 5 * MB + 3 * 16 * 64 * 2 - 2) == ALIAS  # the pool's last element
    assert call(opts=ctypes.byref(sk.LaunchOpts(-2, 0))) == ARG
    if no_device():
        for kw in ({}, dict(out=p + 3 * MB), dict(scales=None), dict(bias=None, res=None), dict(rank=8), dict(rank=128),
                   dict(out=p + 5 * MB + 3 * 16 * 64 * 2)):
            assert call(**kw) == DEVICE, kw


def test_shared_prefix_refusals(lib, mem):
    _, p = mem
    size = lib.skinny_shared_prefix_workspace_bytes(3, 4, 2, 64, 152)
    assert size > 0
    ok = dict(q=p, q_stride=256, rows=3, q_heads=4, prefix_table=p + MB, prefix_width=6, prefix_length=p + MB + 4096,
              block_table=p + 2 * MB, table_stride=4, table_width=4, lengths=p + 3 * MB, scale=0.125, out=p + 4 * MB,
              lse=p + 5 * MB, workspace=p + 8 * MB, workspace_bytes=size)

    def call(cache=None, opts=None, **kw):
        a = sk.SharedPrefixAttentionArgs(**dict(ok, **kw))
        a.cache = cache if cache is not None else cache_at(p + 6 * MB, v=p + 7 * MB)
        return lib.decode_attention_shared_prefix_bf16(bytes(a), opts, None)
    assert lib.decode_attention_shared_prefix_bf16(None, None, None) == NULL
    assert call(cache=cache_at(p, k=None)) == NULL and call(cache=cache_at(p, v=None)) == NULL
    for n in ("q", "prefix_table", "prefix_length", "block_table", "lengths", "out", "workspace"):
        assert call(**{n: None}) == NULL, n
    for kw in (dict(rows=0), dict(rows=1025), dict(q_heads=3), dict(q_heads=0), dict(q_heads=1026),
               dict(table_width=0), dict(table_stride=3), dict(q_stride=248), dict(prefix_width=0),
               dict(prefix_width=-1), dict(prefix_width=1 << 26)):
        assert call(**kw) == SHAPE, kw
    # Key heads * tiles of 64 tokens below 2^31.
    many = cache_at(p + 6 * MB, v=p + 7 * MB, kv_heads=1024, head_stride=0, token_stride=0, page_stride=0)
    assert call(cache=many, rows=1, q_heads=1024, q_stride=1024 * 64, prefix_width=1 << 24) == SHAPE
    for D in (8, 72, 120, 136, 248):
        assert call(cache=cache_at(p + 6 * MB, head_dim=D)) == SHAPE
    for kw in (dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**kw) == ARG, kw
    for kw in (dict(q=p + 8), dict(out=p + 4 * MB + 8), dict(workspace=p + 8 * MB + 8), dict(prefix_table=p + MB + 2),
               dict(prefix_length=p + MB + 4098), dict(block_table=p + 2 * MB + 2), dict(lengths=p + 3 * MB + 2),
               dict(lse=p + 5 * MB + 2), dict(q_stride=260)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(out=p), dict(out=p + MB), dict(out=p + MB + 4096), dict(out=p + 2 * MB), dict(out=p + 3 * MB),
               dict(out=p + 6 * MB), dict(out=p + 7 * MB + 256), dict(lse=p), dict(lse=p + 4 * MB), dict(lse=p + MB + 4096),
               dict(workspace=p + 7 * MB), dict(out=p + 8 * MB + 4096)):
        assert call(**kw) == ALIAS, kw
    assert call(opts=ctypes.byref(sk.LaunchOpts(2, 0))) == ARG
    if no_device():
        for kw in ({}, dict(lse=None), dict(scale=-1.0), dict(prefix_length=p + MB - 4)):
            assert call(**kw) == DEVICE, kw


def test_shared_prefix_workspace_sizes(lib):
    size = lib.skinny_shared_prefix_workspace_bytes
    for bad in ((0, 4, 2, 64, 152), (1025, 4, 2, 64, 152), (3, 4, 0, 64, 152), (3, 3, 2, 64, 152), (3, 0, 1, 64, 152),
                (3, 1026, 1, 64, 152), (3, 4, 2, 72, 152), (3, 4, 2, 64, 0)):
        assert size(*bad) == 0, bad
    for D in (64, 96, 128, 192, 256):
        for group, kv in ((1, 1), (7, 1), (7, 8), (16, 4), (128, 2)):
            last = 0
            for rows in (1, 2, 18, 19, 37, 64, 152, 300, 1024):
                n = size(rows, group * kv, kv, D, 152)
                assert n >= last and n % 16 == 0
                assert n >= lib.skinny_attention_workspace_bytes(152) + rows * group * kv * (D + 1) * 4
                last = n


def test_packed_strings_match_the_structures(lib):
    """The wrappers fill the argument structures as packed strings: the same bytes."""
    n = iter(range(1, 100))
    cache = [next(n) for _ in range(9)]
    first, last = [next(n) for _ in range(4)], [next(n) for _ in range(12)]
    assert bytes(sk.SharedPrefixAttentionArgs(*first, sk.KVCacheArgs(*cache), *last)) == \
        sk._pack_prefix(*first, *cache, *last)
    twelve = [next(n) for _ in range(12)]
    assert bytes(sk.TokenLogprobsArgs(*twelve)) == sk._pack_logprobs(*twelve)
    six = [next(n) for _ in range(6)]
    assert bytes(sk.LoraArgs(*six)) == sk._pack_lora(*six)


def logprobs_call(**kw):
    import torch
    f32, i64 = torch.float32, torch.int64
    a = dict(logits=fake_cuda(3, 100), tokens=fake_cuda(3, 2, dtype=i64), logprobs=fake_cuda(3, 2, dtype=f32),
             entropy=fake_cuda(3, dtype=f32), lse=fake_cuda(3, dtype=f32), top_logprobs=fake_cuda(3, 4, dtype=f32),
             top_tokens=fake_cuda(3, 4, dtype=i64), stream=0)
    a.update(kw)
    return sk.token_logprobs_bf16(**a)


def lora_call(**kw):
    import torch
    a = dict(x=fake_cuda(3, 64), W=fake_cuda(40, 64), out=fake_cuda(3, 40), A=fake_cuda(5, 16, 64),
             B=fake_cuda(5, 40, 16), adapters=fake_cuda(3, dtype=torch.int32), scales=fake_cuda(5, dtype=torch.float32),
             bias=fake_cuda(40), residual=fake_cuda(3, 40), stream=0)
    a.update(kw)
    return sk.decode_gemm_bf16_lora(**a)


def prefix_call(**kw):
    import torch
    i32 = torch.int32
    a = dict(q=fake_cuda(3, 4, 64), k_cache=fake_cuda(4, 16, 2, 64), v_cache=fake_cuda(4, 16, 2, 64),
             prefix_table=fake_cuda(5, dtype=i32), prefix_length=fake_cuda(1, dtype=i32),
             block_table=fake_cuda(3, 4, dtype=i32), lengths=fake_cuda(3, dtype=i32), out=fake_cuda(3, 4, 64),
             lse=fake_cuda(3, 4, dtype=torch.float32), workspace=fake_cuda(64 << 20, dtype=torch.uint8), stream=0)
    a.update(kw)
    return sk.decode_attention_shared_prefix_bf16(**a)


WRAPPERS = [
    (logprobs_call, ["logits", "tokens", "logprobs", "entropy", "lse"]),
    (lora_call, ["x", "W", "out", "A", "B", "adapters", "scales", "bias", "residual"]),
    (prefix_call, ["q", "k_cache", "v_cache", "prefix_table", "prefix_length", "block_table", "lengths", "out", "lse",
                   "workspace"])]


@pytest.mark.parametrize("call,names", WRAPPERS)
def test_what_is_no_tensor_or_of_another_type_is_named(lib, call, names):
    import torch
    for name in names:
        for bad in (3, "x", [1.0]):
            with pytest.raises(TypeError, match=name):
                call(**{name: bad})
        if name != "workspace":
            with pytest.raises(TypeError, match=name):
                call(**{name: fake_cuda(3, 4, dtype=torch.float16)})
            with pytest.raises(ValueError):
                call(**{name: fake_cuda(2, 2, 2, 2, 2, dtype={
                    "tokens": torch.int64, "logprobs": torch.float32, "entropy": torch.float32, "lse": torch.float32,
                    "adapters": torch.int32, "scales": torch.float32, "prefix_table": torch.int32,
                    "prefix_length": torch.int32, "block_table": torch.int32, "lengths": torch.int32}.get(name))})


def test_shapes_that_do_not_fit_are_refused(lib):
    import torch
    f32, i32, i64 = torch.float32, torch.int32, torch.int64
    for call, kw in ((logprobs_call, dict(logits=fake_cuda(4, 100))), (logprobs_call, dict(tokens=None)),
                     (logprobs_call, dict(logprobs=None)), (logprobs_call, dict(logprobs=fake_cuda(3, 3, dtype=f32))),
                     (logprobs_call, dict(tokens=fake_cuda(2, 2, dtype=i64))), (logprobs_call, dict(lse=fake_cuda(4, dtype=f32))),
                     (logprobs_call, dict(top_tokens=fake_cuda(3, 5, dtype=i64))),
                     (logprobs_call, dict(top_logprobs=fake_cuda(4, 4, dtype=f32))),
                     (lora_call, dict(A=fake_cuda(5, 16, 72))), (lora_call, dict(B=fake_cuda(4, 40, 16))),
                     (lora_call, dict(B=fake_cuda(5, 40, 8))), (lora_call, dict(adapters=fake_cuda(4, dtype=i32))),
                     (lora_call, dict(scales=fake_cuda(4, dtype=f32))), (lora_call, dict(W=fake_cuda(40, 72))),
                     (lora_call, dict(residual=fake_cuda(3, 41))), (lora_call, dict(activation="tanh")),
                     (prefix_call, dict(prefix_table=fake_cuda(3, 5, dtype=i32))),
                     (prefix_call, dict(prefix_length=fake_cuda(3, dtype=i32))),
                     (prefix_call, dict(lengths=fake_cuda(1, dtype=i32))),
                     (prefix_call, dict(block_table=fake_cuda(2, 4, dtype=i32))),
                     (prefix_call, dict(out=fake_cuda(3, 4, 32))), (prefix_call, dict(q=fake_cuda(3, 256))),
                     (prefix_call, dict(lse=fake_cuda(3, 2, dtype=f32))), (prefix_call, dict(scale="1"))):
        with pytest.raises(ValueError):
            call(**kw)


def test_calls_with_every_tensor_in_order_reach_the_library(lib):
    if no_device():
        for call in (logprobs_call, lora_call, prefix_call):
            with pytest.raises(sk.SkinnyError) as e:
                call()
            assert e.value.status == DEVICE


def test_the_layer_refuses_options_that_do_not_fit():
    from skinny_bf16_gemm_gb300.layer import DecoderLayer
    plain = [2, 4, 2, 64] + [None] * 16
    for kw in (dict(adapters={"gate": (None, None)}, adapter_ids=0), dict(adapters={"up": (None, None)}),
               dict(prefix_table=0), dict(prefix_length=0), dict(prefix_table=0, prefix_length=0, window=4),
               dict(prefix_table=0, prefix_length=0, sinks=1)):
        with pytest.raises(ValueError):
            DecoderLayer(*plain, **kw)


def test_the_shared_prefix_plan_covers_every_tile_once(tmp_path):
    """tests/native/prefix_plan_check.cpp with the host compiler."""
    import os
    import subprocess
    here = os.path.dirname(os.path.abspath(__file__))
    program = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(sk.PKG, "csrc"), "-x", "c++",
                    os.path.join(here, "native", "prefix_plan_check.cpp"), "-o", program], check=True, timeout=300)
    p = subprocess.run([program], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout == "ok\n", p.stdout
