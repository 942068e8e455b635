"""The decoder-layer operators on the GPU at the edges of what they accept: a single token,
the far ends of the activations, weights that underflow, captures on a given stream."""
import math

import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
import workloads
from attention_helpers import F64, HALF_BF16, check_close
from gpu_helpers import Guarded, gemm_inputs_device
from test_decode_attention_gpu import setup
from test_decoder_layer_gpu import H, build, check_stages, place
from test_epilogue_gpu import extras
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


def attention_calls(n, longest=12000):
    """(arguments, expected output) of n calls whose items span many CTAs."""
    calls = []
    for s in range(n):
        args = setup([longest + 7 * s, 300], 14, 2, 128, 16, seed=40 + s)
        out = torch.empty_like(args[0])
        sk.decode_attention_bf16(*args, out, workspace=sk.attention_workspace())
        calls.append((args, out))
    torch.cuda.synchronize()
    return calls


def test_captured_on_streams_forked_from_the_current_one(cuda_ok):
    """Calls without a workspace on two branches of a capture, while the branch that is the
    current stream takes memory of the workspaces' size and writes over it."""
    calls = attention_calls(3)
    outs = [torch.zeros_like(w) for _, w in calls]
    size = sk.attention_workspace().nbytes
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for _ in range(3):
            for side in sides:
                side.wait_stream(main)
            for side, (args, _), out in zip(sides, calls, outs):
                sk.decode_attention_bf16(*args, out, stream=side)
                torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
            sk.decode_attention_bf16(*calls[2][0], outs[2])
            torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
            for side in sides:
                main.wait_stream(side)
    for _ in range(20):
        for out in outs:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for out, (_, want) in zip(outs, calls):
            assert torch.equal(out, want)


def test_captured_stream_that_is_not_the_current_one(cuda_ok):
    """A graph of calls on its own stream, replayed beside eager calls on that stream and
    beside a second such graph."""
    calls = attention_calls(3)
    outs = [torch.zeros_like(w) for _, w in calls]
    st, other = torch.cuda.Stream(), torch.cuda.Stream()
    sk.decode_attention_bf16(*calls[2][0], outs[2], stream=st)  # the stream's own workspace is there already
    graphs = []
    torch.cuda.synchronize()
    for (args, _), out in zip(calls[:2], outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            with torch.cuda.stream(other):
                sk.decode_attention_bf16(*args, out, stream=st)
        graphs.append(graph)
    lanes = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for lane, graph in zip(lanes, graphs):
            with torch.cuda.stream(lane):
                graph.replay()
        sk.decode_attention_bf16(*calls[2][0], outs[2], stream=st)
        torch.cuda.synchronize()
        for out, (_, want) in zip(outs, calls):
            assert torch.equal(out, want)


def test_given_streams_take_turns_with_the_current_one(cuda_ok):
    """Eager calls on streams given by object and by handle, their workspaces made on the way."""
    calls = attention_calls(3)
    outs = [torch.zeros_like(w) for _, w in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, None]
    for _ in range(20):
        for st, (args, _), out in zip(streams, calls, outs):
            sk.decode_attention_bf16(*args, out, stream=st)
    torch.cuda.synchronize()
    for out, (_, want) in zip(outs, calls):
        assert torch.equal(out, want)
    default = torch.zeros_like(outs[0])
    with torch.cuda.stream(streams[0]):
        sk.decode_attention_bf16(*calls[0][0], default, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(default, calls[0][1])


@pytest.mark.parametrize("M,K", [(1, 8), (16, 7168), (40, 64), (64, 7168)])
@pytest.mark.parametrize("act,lowest", [("silu", -80.0), ("gelu", -12.5), ("gelu_tanh", -10.0)])
def test_activation_tails_keep_their_relative_precision(cuda_ok, M, K, act, lowest):
    """Sums that are the bias exactly (all else is zero), from where a value is about 1e-36 to
    10, every BF16 value on the way: relative to the value, half a BF16 step and what FP32
    leaves of the definition v Phi(v) or v sigmoid(s):
      erf form: v / sqrt 2 is off by 2 U32 at most, by which erfc moves (2 x^2 + 1) times as
      much, x = 12.5 / sqrt 2: 158 * 2 U32; erfc itself 8 steps (16 U32), two products 2 U32:
      below 336 U32 = 2^-15;
      sigmoid forms: s = -2 u to 88, its roundings and its constants' 10 U32 in all, which
      exp multiplies by 88; exp 2 steps, the sum and the quotient 9 U32: below 2^-14."""
    v = torch.arange(0, 2 ** 16, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v) & (v >= lowest) & (v <= 10) & (v.abs() > 1e-30)].contiguous()
    N = v.numel()
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    sk.decode_gemm_bf16_epilogue(x, W, out, v, act)
    d = v.to(F64)
    if act == "gelu":
        want = 0.5 * d * torch.special.erfc(-d / math.sqrt(2))
    else:
        s = d if act == "silu" else 2 * math.sqrt(2 / math.pi) * (d + 0.044715 * d ** 3)
        want = d * torch.sigmoid(s)
    tol = want.abs() * (HALF_BF16 * (1 + 2.0 ** -14) + 2.0 ** -14)
    check_close(out, want.expand(M, N), tol.expand(M, N), act)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_past_their_tails(cuda_ok, act):
    """To the largest finite sums: the sum itself, or next to nothing, never NaN."""
    v = torch.tensor([-3e38, -1e20, -1e13, -500, -120, 0.0, -0.0, 120, 500, 1e13, 1e20, 3e38],
                     device="cuda").to(torch.bfloat16)
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(v.numel(), 8, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(1, v.numel(), dtype=torch.bfloat16, device="cuda")
    sk.decode_gemm_bf16_epilogue(x, W, out, v, act)
    assert torch.equal(out[0], v.clamp(min=0))


@pytest.mark.parametrize("M", [5, 16, 33, 64])
@pytest.mark.parametrize("ragged", [1, 8, 31, 33, 100])
def test_whole_tiles_with_lanes_past_the_right_edge(cuda_ok, M, ragged):
    """The last tile ends inside a warp's 32 columns and takes several rounds of rows: integers,
    bit for bit."""
    N, K = 160 * 128 + ragged, 64
    x, W = gemm_inputs_device(M, N, K, workloads.seed_for("edge", M, N, K), kind="int")
    bias, res = extras(M, N, 9, "int")
    out = Guarded((M, N))
    sk.decode_gemm_bf16_epilogue(x, W, out.tensor, bias, "relu", res)
    torch.cuda.synchronize()
    out.check()
    assert sk.device_error() == (0, 0)
    want = (x.to(F64) @ W.to(F64).t() + bias.to(F64)).clamp(min=0) + res.to(F64)
    assert torch.equal(out.tensor, want.float().to(torch.bfloat16))


def one_token_apart(G, D, n, j, score, value):
    """One row of n tokens of score 0 and small values, token j's score and value given: the
    output of G heads on one key head."""
    page = 16
    g = torch.Generator(device="cuda")
    g.manual_seed(G + D)
    pages = -(-n // page)
    k = torch.zeros(pages, page, 1, D, dtype=torch.bfloat16, device="cuda")
    v = (torch.randn(pages, page, 1, D, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
    k[j // page, j % page, 0, 0] = score
    v[j // page, j % page] = value
    q = torch.zeros(1, G, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out = torch.empty(1, G, D, dtype=torch.bfloat16, device="cuda")
    sk.decode_attention_bf16(q, k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda"), out, scale=1.0)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("G", [1, 16, 32])
def test_weights_that_underflow_add_nothing(cuda_ok, D, G):
    """exp(-300) is 0 in FP32: whatever finite value the token has, the bits are those of a
    value of 0."""
    for n, j in ((40, 7), (700, 650)):
        want = one_token_apart(G, D, n, j, -300.0, 0.0)
        for value in (1.0, 1e30, 3e38, -3e38):
            assert torch.equal(one_token_apart(G, D, n, j, -300.0, value), want)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("G", [1, 16, 32])
def test_small_weights_count(cuda_ok, D, G):
    """A weight of exp(-60) with a value of 2^100 is all of the output but 2^-60 of it; the
    exponent, 87 binary places, is off by 4 roundings of it, 87 * 4 * 2^-24 = 2^-15.6, the
    weight's two terms by 2^-15, the sums by less than 2^-16. A weight above 2^-126 shows an
    infinite value, a weight of exactly 1 too."""
    n, j = 40, 7
    got = one_token_apart(G, D, n, j, -60.0, 2.0 ** 100).to(F64)
    want = torch.full_like(got, math.exp(-60) * 2.0 ** 100 / (n - 1))
    check_close(got, want, want * (HALF_BF16 * 1.01 + 2.0 ** -13), "out")
    for score in (0.0, -60.0, -85.0):
        assert torch.equal(one_token_apart(G, D, n, j, score, math.inf), torch.full_like(want, math.inf).to(torch.bfloat16))
        assert torch.equal(one_token_apart(G, D, n, j, score, -math.inf), torch.full_like(want, -math.inf).to(torch.bfloat16))
