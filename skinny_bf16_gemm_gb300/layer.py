"""One decoder layer for single tokens on the library's calls.

A step takes the residual stream y [M, 7168] of M rows, each the newest token of a
sequence (or one of several drafted tokens: rows that share pages), and returns the
stream after the layer:

    x, res = RMSNorm(y)                          reduce_residual_rmsnorm (one slot)
    qkv    = x Wqkv^T + bqkv                     decode_gemm_bf16_epilogue
    q, cache <- norm, rotate, append             qk_norm_rope_bf16 (q in place in qkv)
    a      = attention(q, cache)                 decode_attention_bf16
    x, res = RMSNorm(sum_r (a Wo^T)_r + res)     decode_gemm_bf16_reduce_rmsnorm
    h      = act(x Wup^T + bup)                  decode_gemm_bf16_epilogue
    y      = h Wdown^T + res                     decode_gemm_bf16_epilogue

Two options serve a batch of many requests. ``adapters``: low-rank adapters of any of the
linears, {"qkv" | "o" | "up" | "down": (A [adapters, rank, K], B [adapters, N, rank])}, with
``adapter_ids`` [M] naming each row's (-1: none) and ``adapter_scales`` [adapters] or None; such
a linear goes by decode_gemm_bf16_lora, and the output linear's reduce and norm by
reduce_residual_rmsnorm. ``prefix_table`` and ``prefix_length``: the pages and the number of
tokens of a prefix that all rows share, by decode_attention_shared_prefix_bf16;
``block_table`` and ``lengths`` are then of the rows' own tokens, and ``positions`` count the
prefix's too.

The attention may be split by heads over tensor-parallel ranks: slots 1.. of ``partials``
then hold the other ranks' rows of the output linear, as in LayerChain. The feed-forward
pair is whole on every rank (W_up, W_down [HIDDEN, F] with all of F): y is the stream
itself, with nothing left to add. The class owns the device buffers and orders the calls on one
stream, optionally as one CUDA graph; the caches, tables, lengths, positions and slots
are the caller's tensors, updated in place between steps.
"""
import torch

from . import (HIDDEN, attention_workspace, decode_attention_bf16, decode_attention_shared_prefix_bf16,
               decode_gemm_bf16_epilogue, decode_gemm_bf16_lora, decode_gemm_bf16_reduce_rmsnorm,
               qk_norm_rope_bf16, reduce_residual_rmsnorm, shared_prefix_workspace)

LINEARS = ("qkv", "o", "up", "down")


class DecoderLayer:
    def __init__(self, M, q_heads, kv_heads, head_dim, W_qkv, W_o, W_up, W_down, gamma_in,
                 gamma_post, q_gamma, k_gamma, rope, k_cache, v_cache, block_table, lengths,
                 positions, slots, b_qkv=None, b_up=None, activation="silu", peers=None, window=0,
                 sinks=0, interleaved=False, eps=1e-6, pdl=True, device="cuda", adapters=None,
                 adapter_ids=None, adapter_scales=None, prefix_table=None, prefix_length=None):
        if any(name not in LINEARS for name in adapters or {}):
            raise ValueError(f"adapters: the linears are {', '.join(LINEARS)}")
        if adapters and adapter_ids is None:
            raise ValueError("adapters need adapter_ids")
        if (prefix_table is None) != (prefix_length is None):
            raise ValueError("prefix_table and prefix_length come together")
        if prefix_table is not None and (window or sinks):
            raise ValueError("a shared prefix has no window")
        self.adapters, self.adapter_ids, self.adapter_scales = dict(adapters or {}), adapter_ids, adapter_scales
        self.prefix_table, self.prefix_length = prefix_table, prefix_length
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.W_qkv, self.W_o, self.W_up, self.W_down = W_qkv, W_o, W_up, W_down
        self.gamma_in, self.gamma_post, self.q_gamma, self.k_gamma = gamma_in, gamma_post, q_gamma, k_gamma
        self.rope, self.k_cache, self.v_cache = rope, k_cache, v_cache
        self.block_table, self.lengths, self.positions, self.slots = block_table, lengths, positions, slots
        self.b_qkv, self.b_up, self.activation = b_qkv, b_up, activation
        self.window, self.sinks, self.interleaved = window, sinks, interleaved
        self.eps, self.pdl = eps, pdl
        bf = dict(dtype=torch.bfloat16, device=device)
        width = q_heads * head_dim
        self.y_in = torch.empty(1, M, HIDDEN, **bf)  # step input, as one partial slot
        self.x = torch.empty(M, HIDDEN, **bf)
        self.res = torch.empty(M, HIDDEN, **bf)
        self.qkv = torch.empty(M, width + 2 * kv_heads * head_dim, **bf)
        self.q = self.qkv[:, :width].view(M, q_heads, head_dim)
        self.attn = torch.empty(M, q_heads, head_dim, **bf)
        self.partials = torch.empty(1 if peers is None else peers.shape[0] + 1, M, HIDDEN, **bf)
        if peers is not None:
            self.partials[1:].copy_(peers)
        self.h = torch.empty(M, W_up.shape[0], **bf)
        self.y = torch.empty(M, HIDDEN, **bf)
        if prefix_table is None:
            self.workspace = attention_workspace(self.x.device)
        else:
            self.workspace = shared_prefix_workspace(M, q_heads, kv_heads, head_dim, self.x.device)
        self.graph = None

    def _linear(self, name, x, W, out, **opts):
        if name not in self.adapters:
            return decode_gemm_bf16_epilogue(x, W, out, **opts)
        A, B = self.adapters[name]
        return decode_gemm_bf16_lora(x, W, out, A, B, self.adapter_ids, scales=self.adapter_scales, **opts)

    def run(self, stream=None):
        """Enqueue one step reading self.y_in; returns the residual stream after the layer."""
        opts = dict(stream=stream, pdl=self.pdl)
        reduce_residual_rmsnorm(self.y_in, None, self.gamma_in, self.x, self.res, self.eps, **opts)
        self._linear("qkv", self.x, self.W_qkv, self.qkv, bias=self.b_qkv, **opts)
        qk_norm_rope_bf16(self.qkv, self.q_heads, self.kv_heads, self.q_gamma, self.k_gamma,
                          self.rope, self.positions, self.q, k_cache=self.k_cache,
                          v_cache=self.v_cache, slots=self.slots, eps=self.eps,
                          interleaved=self.interleaved, **opts)
        if self.prefix_table is None:
            decode_attention_bf16(self.q, self.k_cache, self.v_cache, self.block_table, self.lengths,
                                  self.attn, window=self.window, sinks=self.sinks,
                                  workspace=self.workspace, **opts)
        else:
            decode_attention_shared_prefix_bf16(self.q, self.k_cache, self.v_cache, self.prefix_table,
                                                self.prefix_length, self.block_table, self.lengths,
                                                self.attn, workspace=self.workspace, **opts)
        attn = self.attn.view(self.attn.shape[0], -1)
        if "o" in self.adapters:
            self._linear("o", attn, self.W_o, self.partials[0], **opts)
            reduce_residual_rmsnorm(self.partials, self.res, self.gamma_post, self.x, self.res, self.eps,
                                    **opts)
        else:
            decode_gemm_bf16_reduce_rmsnorm(attn, self.W_o, self.partials, self.res, self.gamma_post,
                                            self.x, self.res, self.eps, **opts)
        self._linear("up", self.x, self.W_up, self.h, bias=self.b_up, activation=self.activation, **opts)
        return self._linear("down", self.h, self.W_down, self.y, residual=self.res, **opts)

    def capture(self):
        """Capture one step as a CUDA graph (after at least one eager step)."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                self.run()
        torch.cuda.current_stream().wait_stream(s)
        self.graph = g
        return self.y

    def replay(self):
        self.graph.replay()
        return self.y
