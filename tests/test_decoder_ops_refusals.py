"""Calls of the decoder-layer operators at the border between accepted and refused, without
a GPU: a call that is accepted gets as far as the missing device."""
import ctypes

import pytest

import skinny_bf16_gemm_gb300 as sk
from test_attention_abi import ALIAS, DEVICE, MB, cache_at, lib, mem, rope_args  # noqa: F401


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
