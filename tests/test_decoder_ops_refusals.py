"""Calls of the decoder-layer operators at the border between accepted and refused, without
a GPU: a call that is accepted gets as far as the missing device."""
import ctypes

import pytest

import skinny_bf16_gemm_gb300 as sk
from test_attention_abi import ALIAS, DEVICE, MB, SHAPE, cache_at, lib, mem, rope_args  # noqa: F401


def accepted(status):
    """The call got past its own checks: host memory is no device memory."""
    return status == DEVICE


@pytest.mark.parametrize("q_stride", [4 * 64, 8 * 64, 5 * 64])
@pytest.mark.parametrize("qkv_stride", [8 * 64, 9 * 64])
def test_one_row_in_place_whatever_the_strides(lib, mem, q_stride, qkv_stride):
    """With one row the distance between rows says nothing: a view of one row has its own
    width there, the rows it is a view of theirs."""
    _, p = mem
    k_heads = p + 4 * 64 * 2

    def call(**kw):
        a = rope_args(p, cache_at(p + 8 * MB), **dict(dict(qkv_stride=qkv_stride, M=1), **kw))
        return lib.qk_norm_rope_bf16(ctypes.byref(a), None, None)
    assert accepted(call(q_out=p, q_stride=q_stride))
    assert accepted(call(k_out=k_heads, k_stride=2 * 64))
    assert accepted(call(q_out=p, q_stride=q_stride, k_out=k_heads, k_stride=3 * 64))
    # Two rows have a distance; other places in the row overlap as before.
    if q_stride != qkv_stride:
        assert call(M=2, q_out=p, q_stride=q_stride) == ALIAS
    assert call(q_out=p + 128, q_stride=q_stride) == ALIAS
    assert call(q_out=k_heads, q_stride=q_stride) == ALIAS
    assert call(q_out=p, q_stride=q_stride, k_out=p, k_stride=2 * 64) == ALIAS


class FakeStreams:
    """The streams of a process without a GPU: a current one, and those being captured."""

    def __init__(self, monkeypatch, current, capturing):
        import contextlib

        import torch
        self.current, self.made = current, []

        @contextlib.contextmanager
        def on(stream):
            before, self.current = self.current, stream
            yield
            self.current = before

        def make(device=None):
            self.made.append(self.current)
            return object()
        for name, f in (("_cuda_getDevice", lambda: 0), ("_cuda_getCurrentRawStream", lambda d: self.current),
                        ("_cuda_isCurrentStreamCapturing", lambda: self.current in capturing)):
            monkeypatch.setattr(torch._C, name, f)
        for name, f in (("stream", on), ("ExternalStream", lambda s, device=None: s),
                        ("default_stream", lambda device=None: 0),
                        ("current_stream", lambda d=None: type("S", (), {"synchronize": lambda s: None})())):
            monkeypatch.setattr(torch.cuda, name, f)
        monkeypatch.setattr(sk, "attention_workspace", make)
        monkeypatch.setattr(sk, "_workspaces", {})

    def workspace(self, stream):
        return sk._own_workspace(0, ctypes.c_void_p(stream))


@pytest.mark.parametrize("capturing", [{11}, {11, 22}, {22}, set()])
def test_a_call_without_workspace_gets_it_on_the_stream_it_runs_on(monkeypatch, capturing):
    """Made and zeroed on the launch stream, so that both come before the kernel and the memory
    is not given to others while it runs; under a capture of that stream, and only then, one
    for the call alone."""
    f = FakeStreams(monkeypatch, 11, capturing)
    a, b = f.workspace(22), f.workspace(22)
    assert f.made == ([22, 22] if 22 in capturing else [22])
    assert (a is b) == (22 not in capturing)
    assert f.current == 11
    f.made.clear()
    a, b = f.workspace(11), f.workspace(11)
    assert f.made == ([11, 11] if 11 in capturing else [11])
    assert (a is b) == (11 not in capturing)
    f.made.clear()
    f.workspace(0)  # the default stream, from another one
    assert f.made == [0]


def test_an_eager_call_after_a_capture_does_not_share_its_workspace(monkeypatch):
    """The graph's workspace is not kept for the stream."""
    capturing = {22}
    f = FakeStreams(monkeypatch, 11, capturing)
    a = f.workspace(22)
    capturing.clear()
    b = f.workspace(22)
    assert a is not b and f.workspace(22) is b


@pytest.mark.parametrize("rows,kv_heads,group,page,tiles16", [
    (1024, 8, 7, 16, (1 << 31) // (1024 * 8)), (64, 1, 1, 1, (1 << 31) // 64), (1024, 2, 100, 32, (1 << 31) // (1024 * 2 * 4))])
def test_most_tokens_of_the_tables(lib, mem, rows, kv_heads, group, page, tiles16):
    """rows * key heads * head blocks * tiles of 16 tokens below 2^31, and a table below 2^30
    tokens: the last width that is accepted, and the first that is not."""
    _, p = mem
    far = 1 << 44  # addresses that are only compared: nothing is read before the device check

    def call(width):
        a = sk.DecodeAttentionArgs(
            q=p, q_stride=kv_heads * group * 64, rows=rows, q_heads=kv_heads * group, block_table=far,
            table_stride=width, table_width=width, lengths=p, scale=1.0, out=far << 1,
            workspace=far << 2, workspace_bytes=1 << 30)
        a.cache = cache_at(p, v=p + MB, page_size=page, kv_heads=kv_heads, num_pages=1, page_stride=0,
                           token_stride=64, head_stride=64)
        return lib.decode_attention_bf16(ctypes.byref(a), None, None)
    tokens = min((tiles16 - 1) * 16, (1 << 30) - 1)
    assert accepted(call(tokens // page))
    assert call(tokens // page + 1) == SHAPE


def fake_cuda(*shape, dtype=None):
    """A host tensor that says it is on a GPU: good for the wrappers' checks only."""
    import torch

    class Fake(torch.Tensor):
        is_cuda = True
    return torch.zeros(shape, dtype=dtype or torch.bfloat16).as_subclass(Fake)


def rope_call(**kw):
    import torch
    a = dict(qkv=fake_cuda(3, 8 * 64), q_heads=4, kv_heads=2, q_gamma=fake_cuda(64), k_gamma=fake_cuda(64),
             rope=fake_cuda(32, 64, dtype=torch.float32), positions=fake_cuda(3, dtype=torch.int32),
             q_out=fake_cuda(3, 4, 64), k_out=fake_cuda(3, 2, 64), k_cache=fake_cuda(4, 16, 2, 64),
             v_cache=fake_cuda(4, 16, 2, 64), slots=fake_cuda(3, dtype=torch.int64), stream=0)
    a.update(kw)
    return sk.qk_norm_rope_bf16(**a)


def attention_call(**kw):
    import torch
    a = dict(q=fake_cuda(3, 4, 64), k_cache=fake_cuda(4, 16, 2, 64), v_cache=fake_cuda(4, 16, 2, 64),
             block_table=fake_cuda(3, 4, dtype=torch.int32), lengths=fake_cuda(3, dtype=torch.int32),
             out=fake_cuda(3, 4, 64), lse=fake_cuda(3, 4, dtype=torch.float32),
             workspace=fake_cuda(64 << 20, dtype=torch.uint8), stream=0)
    a.update(kw)
    return sk.decode_attention_bf16(**a)


@pytest.mark.parametrize("call,names", [
    (rope_call, ["qkv", "q_gamma", "k_gamma", "rope", "positions", "q_out", "k_out", "k_cache", "v_cache", "slots"]),
    (attention_call, ["q", "k_cache", "v_cache", "block_table", "lengths", "out", "lse", "workspace"])])
def test_what_is_no_tensor_is_named(lib, call, names):
    for name in names:
        for bad in (3, "x", [1.0]):
            with pytest.raises(TypeError, match=name):
                call(**{name: bad})


def test_missing_tensors_are_named(lib):
    for name in ("qkv", "positions", "q_out"):
        with pytest.raises(TypeError, match=name):
            rope_call(**{name: None})
    for name in ("q", "k_cache", "v_cache", "block_table", "lengths", "out"):
        with pytest.raises(TypeError, match=name):
            attention_call(**{name: None})
    for name in ("k_cache", "v_cache", "slots"):
        with pytest.raises(ValueError, match="go together"):
            rope_call(**{name: None})


def test_tensors_without_axes_and_numbers_out_of_range(lib):
    import torch
    for name in ("qkv", "q_out", "k_out", "rope", "positions", "slots", "k_cache"):
        with pytest.raises(ValueError, match=name):
            rope_call(**{name: fake_cuda(dtype={"rope": torch.float32, "positions": torch.int32,
                                                "slots": torch.int64}.get(name))})
    for name in ("q", "out", "block_table", "lengths", "k_cache"):
        with pytest.raises(ValueError, match=name):
            attention_call(**{name: fake_cuda(dtype={"block_table": torch.int32, "lengths": torch.int32}.get(name))})
    for kw in (dict(window=1 << 31), dict(sinks=1 << 40), dict(window=1.5), dict(scale="1")):
        with pytest.raises(ValueError, match="decode_attention_bf16"):
            attention_call(**kw)
    with pytest.raises(ValueError, match="qk_norm_rope_bf16"):
        rope_call(eps="1")


def test_calls_with_every_tensor_in_order_reach_the_library(lib):
    for call in (rope_call, attention_call):
        with pytest.raises(sk.SkinnyError) as e:
            call()
        assert accepted(e.value.status)


def elements(page, token, head, sizes, D, base=0):
    """Every element that a pool's keys (or values) touch, in 8-element chunks."""
    return [base + i * page + j * token + h * head + c
            for i in range(sizes[0]) for j in range(sizes[1]) for h in range(sizes[2]) for c in range(0, D, 8)]


def test_pools_whose_elements_meet_are_refused_for_writing(lib, mem):
    """Seeded small layouts, by enumeration: a pool that would store two elements in one place
    is refused; one whose axes lie within each other is accepted."""
    import random
    _, p = mem
    r = random.Random(4)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        D = 8 * r.choice([1, 2, 3])
        sizes = [r.choice([1, 2, 3, 4]) for _ in range(3)]
        order = r.sample(range(3), 3)
        strides, extent = [0, 0, 0], D
        for axis in order:  # innermost first, padded now and then, sometimes too near
            strides[axis] = extent + 8 * r.choice([0, 0, 0, 1, 5]) - 8 * r.choice([0, 0, 0, 0, 0, 1, 2])
            extent += strides[axis] * (sizes[axis] - 1) + r.choice([0, 0, D])
        if any(n > 1 and s < D for n, s in zip(sizes, strides)):
            continue
        gap = 8 * r.choice([1, D // 8, strides[order[0]] // 8, extent // 8, extent // 8 + 3, r.randint(1, extent // 4)])
        gap *= r.choice([1, -1])
        base = p + 8 * MB
        cache = cache_at(base, v=base + 2 * gap, num_pages=sizes[0], page_size=sizes[1], kv_heads=sizes[2],
                         head_dim=D, page_stride=strides[0], token_stride=strides[1], head_stride=strides[2])
        a = rope_args(p, cache, kv_heads=sizes[2], head_dim=D, rot_dim=0, k_out=None)
        got = lib.qk_norm_rope_bf16(ctypes.byref(a), None, None)
        if min(strides) < 0:
            assert got == SHAPE
            continue
        k = elements(*strides, sizes, D)
        kv = k + [e + gap for e in k]
        meets = len(set(kv)) < len(kv)
        nested, end = True, D
        for s, n in sorted((s, n) for s, n in zip(strides, sizes) if n > 1):
            nested, end = nested and s >= end, end + s * (n - 1)
        if meets:
            assert got == ALIAS, (sizes, strides, D, gap)
        elif nested:
            assert accepted(got), (sizes, strides, D, gap)
        seen[meets] += 1
    assert min(seen.values()) > 500


def test_pools_only_read_may_repeat(lib, mem):
    """Keys and values that are only read may lie anywhere: one head's for all, a page's for all."""
    _, p = mem
    for kw in (dict(head_stride=0), dict(page_stride=0), dict(token_stride=0), dict(v=p + 6 * MB)):
        a = sk.DecodeAttentionArgs(q=p, q_stride=256, rows=3, q_heads=4, block_table=p + 2 * MB, table_stride=4,
                                   table_width=4, lengths=p + 3 * MB, scale=0.125, out=p + 4 * MB,
                                   workspace=p + 8 * MB, workspace_bytes=64 << 20)
        a.cache = cache_at(p + 6 * MB, **dict(dict(v=p + 7 * MB), **kw))
        assert accepted(lib.decode_attention_bf16(ctypes.byref(a), None, None))


def test_most_rows_of_the_rotation(lib, mem):
    """Rows are numbered in 32 bits, and the rows after the next one with them."""
    far = 1 << 40  # addresses that are only compared

    def call(M):
        a = sk.QkNormRopeArgs(qkv=far, qkv_stride=24, M=M, q_heads=1, kv_heads=1, head_dim=8, eps=1e-6,
                              q_out=far << 1, q_stride=8)
        return lib.qk_norm_rope_bf16(ctypes.byref(a), None, None)
    assert accepted(call(1 << 30))
    assert call((1 << 30) + 1) == SHAPE and call((1 << 31) - 1) == SHAPE
