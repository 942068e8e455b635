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

The attention may be split by heads over tensor-parallel ranks: slots 1.. of ``partials``
then hold the other ranks' rows of the output linear, as in LayerChain. The feed-forward
pair is whole on every rank (W_up, W_down [HIDDEN, F] with all of F): y is the stream
itself, with nothing left to add. The class owns the device buffers and orders the calls on one
stream, optionally as one CUDA graph; the caches, tables, lengths, positions and slots
are the caller's tensors, updated in place between steps.
"""
import torch

from . import (HIDDEN, attention_workspace, decode_attention_bf16, decode_gemm_bf16_epilogue,
               decode_gemm_bf16_reduce_rmsnorm, qk_norm_rope_bf16, reduce_residual_rmsnorm)


class DecoderLayer:
    def __init__(self, M, q_heads, kv_heads, head_dim, W_qkv, W_o, W_up, W_down, gamma_in,
                 gamma_post, q_gamma, k_gamma, rope, k_cache, v_cache, block_table, lengths,
                 positions, slots, b_qkv=None, b_up=None, activation="silu", peers=None, window=0,
                 sinks=0, interleaved=False, eps=1e-6, pdl=True, device="cuda"):
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
        self.workspace = attention_workspace(self.x.device)
        self.graph = None

    def run(self, stream=None):
        """Enqueue one step reading self.y_in; returns the residual stream after the layer."""
        opts = dict(stream=stream, pdl=self.pdl)
        reduce_residual_rmsnorm(self.y_in, None, self.gamma_in, self.x, self.res, self.eps, **opts)
        decode_gemm_bf16_epilogue(self.x, self.W_qkv, self.qkv, bias=self.b_qkv, **opts)
        qk_norm_rope_bf16(self.qkv, self.q_heads, self.kv_heads, self.q_gamma, self.k_gamma,
                          self.rope, self.positions, self.q, k_cache=self.k_cache,
                          v_cache=self.v_cache, slots=self.slots, eps=self.eps,
                          interleaved=self.interleaved, **opts)
        decode_attention_bf16(self.q, self.k_cache, self.v_cache, self.block_table, self.lengths,
                              self.attn, window=self.window, sinks=self.sinks,
                              workspace=self.workspace, **opts)
        decode_gemm_bf16_reduce_rmsnorm(self.attn.view(self.attn.shape[0], -1), self.W_o,
                                        self.partials, self.res, self.gamma_post, self.x, self.res,
                                        self.eps, **opts)
        decode_gemm_bf16_epilogue(self.x, self.W_up, self.h, bias=self.b_up,
                                  activation=self.activation, **opts)
        return decode_gemm_bf16_epilogue(self.h, self.W_down, self.y, residual=self.res, **opts)

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
