"""A decode step of a batch of requests as a server runs it: a decoder layer whose rows have
adapters of their own behind a prefix that all share, the logits of its output, and what is
sampled and reported from them. Every stage against 64 bits on the inputs that it had; over
several steps that feed the likeliest tokens back, eager, with PDL and replayed as a graph."""
import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
from skinny_bf16_gemm_gb300.layer import DecoderLayer
from attention_helpers import F64, HALF_BF16, check_close, norm_rope_reference
from test_decoder_layer_gpu import build
from test_lora_gpu import reference as lora_reference
from test_shared_prefix_gpu import reference as prefix_reference
from test_token_logprobs_gpu import reference as logprobs_reference

pytestmark = pytest.mark.gpu
H, V, TOP = sk.HIDDEN, 5003, 4


class Server:
    """A layer, an embedding that is the output matrix too, and the step's buffers."""

    def __init__(self, names, M=6, Hq=14, Hkv=2, D=128, F=2048, prefix=285, pdl=True, peers=True, seed=0, rank=16):
        base, self.randn = build(M=M, Hq=Hq, Hkv=Hkv, D=D, F=F, pages=6 * M, pdl=pdl, peers=peers, seed=seed)
        b, randn = base, self.randn
        widths = dict(qkv=b.W_qkv.shape, o=b.W_o.shape, up=b.W_up.shape, down=b.W_down.shape)
        adapters = {n: (randn(5, rank, widths[n][1], std=widths[n][1] ** -0.5), randn(5, widths[n][0], rank, std=rank ** -0.5))
                    for n in names}
        ids = torch.tensor([4, -1, 2, 2, 0, 1] * M, dtype=torch.int32, device="cuda")[:M]
        scales = torch.tensor([0.5, 1.0, 2.0, 0.25, 1.5], device="cuda")
        # Three pages a row for its own tokens, the others for the prefix.
        table = b.block_table[:, :3].contiguous()
        prefix_table = b.block_table[:, 3:].reshape(-1).contiguous()
        self.prefix = prefix
        self.layer = DecoderLayer(
            M, Hq, Hkv, D, b.W_qkv, b.W_o, b.W_up, b.W_down, b.gamma_in, b.gamma_post, b.q_gamma, b.k_gamma, b.rope,
            b.k_cache, b.v_cache, table, b.lengths, b.positions, b.slots, b_qkv=b.b_qkv, b_up=b.b_up,
            activation="gelu_tanh", peers=b.partials[1:] if peers else None, pdl=pdl, adapters=adapters,
            adapter_ids=ids if names else None, adapter_scales=scales if names else None, prefix_table=prefix_table,
            prefix_length=torch.tensor([prefix], dtype=torch.int32, device="cuda"))
        self.pdl, self.M = pdl, M
        self.head = randn(V, H, std=H ** -0.5)
        self.logits = torch.empty(M, V, dtype=torch.bfloat16, device="cuda")
        self.tokens = (torch.arange(M, device="cuda") * 700 + 3) % V
        self.logprobs = torch.empty(M, device="cuda")
        self.entropy, self.lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        self.top_logprobs = torch.empty(M, TOP, device="cuda")
        self.top_tokens = torch.zeros(M, TOP, dtype=torch.int64, device="cuda")

    def place(self, own):
        """Row r's new token the own[r]-th of its own tokens (-1: padding)."""
        assert self.prefix + max(own) < self.layer.rope.shape[0] and max(own) < 3 * self.layer.k_cache.shape[1]
        layer, page = self.layer, self.layer.k_cache.shape[1]
        for r, p in enumerate(own):
            layer.positions[r] = self.prefix + max(p, 0)
            layer.lengths[r] = p + 1
            layer.slots[r] = int(layer.block_table[r, p // page]) * page + p % page if p >= 0 else -1

    def run(self):
        layer = self.layer
        layer.y_in[0].copy_(self.head[self.tokens] * 40)
        y = layer.run()
        sk.decode_gemm_bf16_logits(y, self.head, self.logits)
        sk.token_logprobs_bf16(self.logits, self.tokens, self.logprobs, self.entropy, self.lse, self.top_logprobs,
                               self.top_tokens, pdl=self.pdl)

    def feed_back(self):
        self.tokens.copy_(self.top_tokens[:, 0])


def linear(layer, name, x, W, bias=None, act="none", residual=None):
    """(want, tolerance) of one of the layer's linears in 64 bits."""
    A, B = layer.adapters.get(name, (torch.zeros(1, 8, W.shape[1], dtype=torch.bfloat16, device="cuda"),
                                     torch.zeros(1, W.shape[0], 8, dtype=torch.bfloat16, device="cuda")))
    ids = layer.adapter_ids if name in layer.adapters else torch.full((x.shape[0],), -1)
    return lora_reference(x, W, A, B, ids, layer.adapter_scales if name in layer.adapters else None, bias, act, residual)


def check_step(s):
    layer, M = s.layer, s.M
    y_in = layer.y_in[0]
    x1, r1 = torch.empty_like(layer.x), torch.empty_like(layer.res)
    sk.reduce_residual_rmsnorm(layer.y_in, None, layer.gamma_in, x1, r1, 1e-6)
    assert torch.equal(r1, y_in)
    Hq, Hkv, D = layer.q_heads, layer.kv_heads, layer.head_dim
    qkv = torch.empty_like(layer.qkv)
    layer._linear("qkv", x1, layer.W_qkv, qkv, bias=layer.b_qkv)
    check_close(qkv, *linear(layer, "qkv", x1, layer.W_qkv, layer.b_qkv), "qkv")
    heads = qkv.view(M, Hq + 2 * Hkv, D)
    check_close(layer.q, *norm_rope_reference(heads[:, :Hq], layer.q_gamma, layer.rope, layer.positions, False, 1e-6), "q")
    page = layer.k_cache.shape[1]
    for r, at in enumerate(layer.slots.tolist()):
        if at >= 0:
            assert torch.equal(layer.v_cache[at // page, at % page], heads[r, Hq + Hkv:])
    want, _, tol, _ = prefix_reference(layer.q, layer.k_cache, layer.v_cache, layer.prefix_table, s.prefix,
                                       layer.block_table, layer.lengths, D ** -0.5)
    check_close(layer.attn, want, tol, "attention")
    attn = layer.attn.view(M, -1)
    check_close(layer.partials[0], *linear(layer, "o", attn, layer.W_o), "output linear")
    x2, r2 = torch.empty_like(x1), torch.empty_like(r1)
    sk.reduce_residual_rmsnorm(layer.partials, r1, layer.gamma_post, x2, r2, 1e-6)
    assert torch.equal(layer.x, x2) and torch.equal(layer.res, r2)
    check_close(layer.h, *linear(layer, "up", x2, layer.W_up, layer.b_up, "gelu_tanh"), "up")
    check_close(layer.y, *linear(layer, "down", layer.h, layer.W_down, residual=r2), "down")
    logits = layer.y.to(F64) @ s.head.to(F64).t()
    e = (H / 16 + 16) * 2.0 ** -23 * (layer.y.to(F64).abs() @ s.head.to(F64).abs().t())
    check_close(s.logits, logits, e + HALF_BF16 * (logits.abs() + e), "logits")
    want, order = logprobs_reference(s.logits, s.tokens[:, None], TOP)
    for name, (w, tol) in want.items():
        check_close(getattr(s, name).view_as(w), w, tol, name)
    assert torch.equal(s.top_tokens, order)


@pytest.mark.parametrize("pdl", [False, True])
@pytest.mark.parametrize("names", [(), ("qkv", "o", "up", "down"), ("qkv", "down"), ("o",)])
def test_steps_of_a_batch(cuda_ok, names, pdl):
    s = Server(names, pdl=pdl)
    start = [0, 15, 40, 27, -1, 7]
    for step in range(3):
        s.place([p + step if p >= 0 else -1 for p in start])
        s.run()
        torch.cuda.synchronize()
        assert sk.device_error() == (0, 0)
        check_step(s)
        s.feed_back()


def test_a_full_batch_of_high_rank(cuda_ok):
    """60 rows: the prefix is read once, the adapters' second factors by way of shared memory."""
    s = Server(("qkv", "o", "up", "down"), M=60, Hq=16, Hkv=2, prefix=440, rank=64, seed=5)
    s.place([(7 * r) % 40 for r in range(60)])
    s.run()
    torch.cuda.synchronize()
    assert sk.device_error() == (0, 0)
    check_step(s)


def test_replayed_steps_equal_eager_ones(cuda_ok):
    names = ("qkv", "o", "up", "down")
    eager, graph = Server(names, seed=3), Server(names, seed=3)
    start = [3, 16, 31, 9, -1, 20]
    first = graph.tokens.clone()
    graph.place(start)
    graph.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.run()
    graph.tokens.copy_(first)
    graph.layer.k_cache.copy_(eager.layer.k_cache)
    graph.layer.v_cache.copy_(eager.layer.v_cache)
    for step in range(4):
        for s in (eager, graph):
            s.place([p + step if p >= 0 else -1 for p in start])
        eager.run()
        g.replay()
        torch.cuda.synchronize()
        assert sk.device_error() == (0, 0)
        for name in ("logits", "logprobs", "entropy", "lse", "top_logprobs", "top_tokens"):
            assert torch.equal(getattr(eager, name), getattr(graph, name)), name
        assert torch.equal(eager.layer.k_cache, graph.layer.k_cache)
        eager.feed_back()
        graph.feed_back()


def test_a_layer_without_the_options_keeps_its_bits(cuda_ok):
    """A shared prefix and the same tokens in every row's own table; no adapter in use."""
    s = Server(("up",), seed=7, prefix=288)
    s.layer.adapter_ids.fill_(-1)
    s.place([5, 20, 0, 33, 40, 7])
    s.run()
    base, _ = build(M=6, pages=36, seed=7)
    b, layer = base, s.layer
    b.block_table = torch.cat([layer.prefix_table[None].expand(6, -1), layer.block_table], 1).contiguous()
    b.lengths, b.positions, b.slots = layer.lengths + 288, layer.positions, layer.slots
    b.y_in[0].copy_(layer.y_in[0])
    b.k_cache.copy_(layer.k_cache)
    b.v_cache.copy_(layer.v_cache)
    b.run()
    torch.cuda.synchronize()
    assert torch.equal(b.q, layer.q)
    assert (b.attn.float() - layer.attn.float()).abs().max() < 0.02
    h = torch.empty_like(layer.h)
    sk.decode_gemm_bf16_epilogue(layer.x, layer.W_up, h, bias=layer.b_up, activation="gelu_tanh")
    assert torch.equal(h, layer.h)
