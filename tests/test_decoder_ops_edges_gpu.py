"""The decoder-layer operators on the GPU at the edges of what they accept: a single token,
the far ends of the activations, weights that underflow, captures on a given stream."""
import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
from test_decoder_layer_gpu import H, build, check_stages, place
from test_qk_norm_rope_gpu import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(7, 1, 128), (56, 8, 128), (3, 2, 96)])
@pytest.mark.parametrize("pad", [0, 40])
def test_one_row_rotated_in_place(cuda_ok, Hq, Hkv, D, pad):
    qkv, qg, kg, rope, pos = inputs(1, Hq, Hkv, D, D)
    q, k = torch.empty(1, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(
        1, Hkv, D, dtype=torch.bfloat16, device="cuda")
    sk.qk_norm_rope_bf16(qkv, Hq, Hkv, qg, kg, rope, pos, q, k)
    wide = torch.full((1, qkv.shape[1] + 2 * pad), 3.0, dtype=torch.bfloat16, device="cuda")
    row = wide[:, pad:pad + qkv.shape[1]]
    row.copy_(qkv)
    qv, kv = row[:, :Hq * D].view(1, Hq, D), row[:, Hq * D:(Hq + Hkv) * D].view(1, Hkv, D)
    sk.qk_norm_rope_bf16(row, Hq, Hkv, qg, kg, rope, pos, qv, kv)
    torch.cuda.synchronize()
    assert torch.equal(qv, q) and torch.equal(kv, k)
    assert torch.equal(row[:, (Hq + Hkv) * D:], qkv[:, (Hq + Hkv) * D:])
    assert (wide[:, :pad] == 3).all() and (wide[:, pad + qkv.shape[1]:] == 3).all()


@pytest.mark.parametrize("pdl", [False, True])
def test_layer_of_one_token(cuda_ok, pdl):
    """Steps of a single sequence, eager and as a graph."""
    layer, randn = build(M=1, Hq=7, Hkv=1, pages=20, pdl=pdl)
    for step in range(3):
        y_in = randn(1, H)
        layer.y_in[0].copy_(y_in)
        place(layer, [15 + step])
        layer.run()
        torch.cuda.synchronize()
        assert sk.device_error() == (0, 0)
        check_stages(layer, y_in)
    layer.capture()
    y_in = randn(1, H)
    layer.y_in[0].copy_(y_in)
    place(layer, [18])
    layer.replay()
    torch.cuda.synchronize()
    check_stages(layer, y_in)
