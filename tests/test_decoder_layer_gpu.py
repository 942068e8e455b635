"""The decoder layer: the new operators together with the ones they stand beside, as a
user runs them. Each stage against its definition in 64 bits on its own inputs, over
several tokens that grow the cache, eager, with PDL and replayed as a graph."""
import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
from skinny_bf16_gemm_gb300.layer import DecoderLayer
from attention_helpers import F64, HALF_BF16, attention_reference, check_close, norm_rope_reference, rope_table

pytestmark = pytest.mark.gpu
H = sk.HIDDEN


def build(M=6, Hq=14, Hkv=2, D=128, F=2048, page=16, pages=40, window=0, sinks=0, pdl=True, peers=True, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(torch.bfloat16)
    W = (Hq + 2 * Hkv) * D
    width = pages // M
    table = torch.randperm(pages, generator=g, device="cuda")[:M * width].view(M, width).to(torch.int32)
    layer = DecoderLayer(
        M, Hq, Hkv, D, randn(W, H, std=H ** -0.5), randn(H, Hq * D, std=(Hq * D) ** -0.5),
        randn(F, H, std=H ** -0.5), randn(H, F, std=F ** -0.5), randn(H, std=0.1, mean=1), randn(H, std=0.1, mean=1),
        randn(D, std=0.1, mean=1), randn(D, std=0.1, mean=1), rope_table(512, D),
        randn(pages, page, Hkv, D), randn(pages, page, Hkv, D), table,
        torch.zeros(M, dtype=torch.int32, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda"),
        torch.zeros(M, dtype=torch.int64, device="cuda"), b_qkv=randn(W, std=0.2), b_up=randn(F, std=0.2),
        activation="gelu_tanh", peers=randn(3, M, H) if peers else None, window=window, sinks=sinks, pdl=pdl)
    return layer, randn


def place(layer, pos):
    """Row r's new token at pos[r] (-1: padding)."""
    page = layer.k_cache.shape[1]
    for r, p in enumerate(pos):
        layer.positions[r] = max(p, 0)
        layer.lengths[r] = p + 1
        layer.slots[r] = int(layer.block_table[r, p // page]) * page + p % page if p >= 0 else -1


def check_stages(layer, y_in):
    """Every stage's output against 64 bits on the inputs that the stage had."""
    M = y_in.shape[0]
    x = y_in.to(F64)
    norm = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * layer.gamma_in.to(F64)
    xb = norm.to(torch.bfloat16)
    # The layer's buffers hold later stages' values, so the first stages are made again by calls of their own.
    x1, r1 = torch.empty(M, H, dtype=torch.bfloat16, device="cuda"), torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    sk.reduce_residual_rmsnorm(y_in[None].contiguous(), None, layer.gamma_in, x1, r1, 1e-6)
    check_close(x1, norm, HALF_BF16 * norm.abs() * 1.01 + 1e-6, "norm")
    assert torch.equal(r1, y_in) and xb.shape == x1.shape
    qkv = torch.empty_like(layer.qkv)
    sk.decode_gemm_bf16_epilogue(x1, layer.W_qkv, qkv, bias=layer.b_qkv)
    Hq, Hkv, D = layer.q_heads, layer.kv_heads, layer.head_dim
    heads = qkv.view(M, Hq + 2 * Hkv, D)
    want, tol = norm_rope_reference(heads[:, :Hq], layer.q_gamma, layer.rope, layer.positions, False, 1e-6)
    check_close(layer.q, want, tol, "q")
    want_k, tol_k = norm_rope_reference(heads[:, Hq:Hq + Hkv], layer.k_gamma, layer.rope, layer.positions, False, 1e-6)
    page = layer.k_cache.shape[1]
    for r, s in enumerate(layer.slots.tolist()):
        if s >= 0:
            check_close(layer.k_cache[s // page, s % page], want_k[r], tol_k[r], "cached key")
            assert torch.equal(layer.v_cache[s // page, s % page], heads[r, Hq + Hkv:])
    want, _, tol, _ = attention_reference(layer.q, layer.k_cache, layer.v_cache, layer.block_table, layer.lengths,
                                          D ** -0.5, layer.window, layer.sinks)
    check_close(layer.attn, want, tol, "attention")
    # Output linear, reduce and norm, and the feed-forward pair by their plain calls, bit for bit.
    part = layer.partials.clone()
    sk.decode_gemm_bf16(layer.attn.view(M, -1), layer.W_o, part[0])
    x2, r2 = torch.empty_like(x1), torch.empty_like(x1)
    sk.reduce_residual_rmsnorm(part, r1, layer.gamma_post, x2, r2, 1e-6)
    assert torch.equal(layer.x, x2) and torch.equal(layer.res, r2)
    h = x2.to(F64) @ layer.W_up.to(F64).t() + layer.b_up.to(F64)
    h = 0.5 * h * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (h + 0.044715 * h ** 3)))
    e = (H / 16 + 16) * 2.0 ** -23 * (x2.abs().to(F64) @ layer.W_up.abs().to(F64).t())
    check_close(layer.h, h, 1.13 * e + 2.0 ** -19 + HALF_BF16 * (h.abs() + 1.13 * e), "up")
    y = layer.h.to(F64) @ layer.W_down.to(F64).t() + r2.to(F64)
    F = layer.h.shape[1]
    e = (F / 16 + 16) * 2.0 ** -23 * (layer.h.abs().to(F64) @ layer.W_down.abs().to(F64).t())
    check_close(layer.y, y, e + 2.0 ** -22 * y.abs() + HALF_BF16 * (y.abs() + e), "down")


@pytest.mark.parametrize("pdl", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 2)])
def test_steps_grow_the_cache(cuda_ok, pdl, window, sinks):
    layer, randn = build(pdl=pdl, window=window, sinks=sinks)
    start = [0, 15, 40, 70, -1, 7]
    for step in range(4):
        y_in = randn(6, H)
        layer.y_in[0].copy_(y_in)
        place(layer, [p + step if p >= 0 else -1 for p in start])
        layer.run()
        torch.cuda.synchronize()
        assert sk.device_error() == (0, 0)
        check_stages(layer, y_in)
        assert not layer.attn[4].any()


def test_drafted_tokens_of_one_sequence(cuda_ok):
    """Rows 0..3: four drafted tokens of one sequence in one step. Each row's key is in the
    cache before any row reads it, and a row sees its own and the earlier ones only."""
    layer, randn = build(M=4, pages=40, peers=False)
    layer.block_table.copy_(layer.block_table[:1].expand(4, -1).contiguous())
    y_in = randn(4, H)
    layer.y_in[0].copy_(y_in)
    place(layer, [30, 31, 32, 33])
    layer.run()
    torch.cuda.synchronize()
    check_stages(layer, y_in)


def test_graph_replays_equal_eager_steps(cuda_ok):
    eager, randn = build(seed=3)
    graph, _ = build(seed=3)
    start = [3, 16, 31, 90, -1, 50]
    place(graph, start)
    graph.y_in.zero_()
    graph.run()
    graph.capture()
    # The warm-up steps wrote the first tokens' keys; put both caches in the same state.
    graph.k_cache.copy_(eager.k_cache)
    graph.v_cache.copy_(eager.v_cache)
    for step in range(5):
        y_in = randn(6, H)
        for layer in (eager, graph):
            layer.y_in[0].copy_(y_in)
            place(layer, [p + step if p >= 0 else -1 for p in start])
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.y, graph.y)
        assert torch.equal(eager.k_cache, graph.k_cache) and torch.equal(eager.v_cache, graph.v_cache)


def test_two_layers_keep_the_plain_calls_bits(cuda_ok):
    """Layers back to back with PDL give the bits of the same calls made one by one
    without it."""
    layers = [build(seed=s)[0] for s in (5, 6)]
    twins = [build(seed=s, pdl=False)[0] for s in (5, 6)]
    _, randn = build(seed=7)
    y_in = randn(6, H)
    pos = [5, 20, 33, 64, 80, 95]
    ends = []
    for pair in (layers, twins):
        y = y_in
        for layer in pair:
            place(layer, pos)
        torch.cuda.synchronize()
        for layer in pair:
            layer.y_in[0].copy_(y)
            y = layer.run()
            if pair is twins:
                torch.cuda.synchronize()
        ends.append(y)
    torch.cuda.synchronize()
    assert torch.equal(*ends)


FIRST_CALLS_CAPTURED = """
import torch, skinny_bf16_gemm_gb300 as sk
D = 128
qkv = torch.randn(3, 9 * D, device="cuda").bfloat16()
gamma = torch.ones(D, device="cuda").bfloat16()
rope = torch.randn(100, D, device="cuda")
pos = torch.zeros(3, dtype=torch.int32, device="cuda")
q = torch.empty(3, 7, D, device="cuda", dtype=torch.bfloat16)
k = torch.randn(10, 16, 1, D, device="cuda").bfloat16()
v = k.clone()
slots = torch.arange(3, device="cuda")
table = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
lengths = torch.tensor([40, 3, 20], dtype=torch.int32, device="cuda")
out = torch.zeros_like(q)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    sk.qk_norm_rope_bf16(qkv, 7, 1, gamma, gamma, rope, pos, q, k_cache=k, v_cache=v, slots=slots)
    sk.decode_attention_bf16(q, k, v, table, lengths, out)
graph.replay()
torch.cuda.synchronize()
replayed = out.clone()
sk.decode_attention_bf16(q, k, v, table, lengths, out)
assert torch.equal(replayed, out) and out.any() and sk.device_error() == (0, 0)
print("ok")
"""


def test_first_calls_of_a_process_captured(cuda_ok):
    """Rotation and attention may be captured from a process's first call on."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], capture_output=True, text=True, cwd=root,
                       timeout=300)
    assert p.returncode == 0 and "ok" in p.stdout, p.stderr
