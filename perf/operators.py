"""The operators of a decoder layer for single tokens, as measured cases.

  epilogue   decode_gemm_bf16_epilogue: out = act(x W^T + bias) + residual
  rope       qk_norm_rope_bf16: RMSNorm of every query and key head, position rotation,
             and the append of keys and values to a paged cache
  attention  decode_attention_bf16: one new token per row over a paged cache, with an
             optional sliding window and always-visible first tokens

``own`` false: run() computes them with elementary torch operations in 32 bits, rounded
once at the end. ``own`` true: run() calls the framework. exact() has them in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # One drafted token through a small projection with an activation: latency.
        dict(name="epilogue 1x2048x7168 silu", op="epilogue", M=1, N=2048, K=7168, act="silu",
             bias=True, residual=False),
        # Ragged everything: odd rows, an odd output width, K that ends inside a block.
        dict(name="epilogue 5x4099x1000 relu res", op="epilogue", M=5, N=4099, K=1000, act="relu",
             bias=True, residual=True),
        # The chain's up linear with its activation at the chain's 16 rows.
        dict(name="epilogue 16x18432x7168 gelu", op="epilogue", M=16, N=18432, K=7168,
             act="gelu_tanh", bias=True, residual=False),
        # The chain's down linear at the row cap, adding the residual stream.
        dict(name="epilogue 64x7168x18432 res", op="epilogue", M=64, N=7168, K=18432, act="none",
             bias=True, residual=True),
        # One token of one tensor-parallel rank (7 query heads, 1 key head): latency.
        dict(name="rope 1 row 7+1 heads", op="rope", M=1, Hq=7, Hkv=1, D=128, rot=128, page=16,
             interleaved=False, hnd=False),
        # A decode batch at the row cap, all heads of a 7168-wide layer on one GPU.
        dict(name="rope 64 rows 56+8 heads", op="rope", M=64, Hq=56, Hkv=8, D=128, rot=128, page=16,
             interleaved=False, hnd=False),
        # A prompt's tokens into the cache: half the head rotated, interleaved pairs.
        dict(name="rope 8191 rows prompt", op="rope", M=8191, Hq=56, Hkv=8, D=128, rot=64, page=64,
             interleaved=True, hnd=True),
        # The first steps after a short prompt, one rank's heads: latency.
        dict(name="attention 1 row 129", op="attention", R=1, Hq=7, Hkv=1, D=128, longest=129,
             ragged=False, page=16, window=0, sinks=0, hnd=False),
        # A ragged decode batch of one rank, some rows empty (padding) or one token long.
        dict(name="attention 64 ragged to 4000", op="attention", R=64, Hq=7, Hkv=1, D=128,
             longest=4000, ragged=True, page=16, window=0, sinks=0, hnd=False),
        # One user with a long context: all parallelism comes from the split over the length.
        dict(name="attention 1 row 131071", op="attention", R=1, Hq=56, Hkv=8, D=128,
             longest=131071, ragged=False, page=64, window=0, sinks=0, hnd=False),
        # Long chats under a sliding window with four sinks: only what is visible is read.
        dict(name="attention 32 window 4096", op="attention", R=32, Hq=56, Hkv=8, D=128,
             longest=20000, ragged=True, page=32, window=4096, sinks=4, hnd=True),
        # A full serving batch, small heads in groups of four.
        dict(name="attention 64 ragged to 16384", op="attention", R=64, Hq=32, Hkv=8, D=64,
             longest=16384, ragged=True, page=16, window=0, sinks=0, hnd=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["epilogue", "rope", "attention"])
    if op == "epilogue":
        N = _log(rng, 100, 20480)
        return dict(op=op, M=rng.randint(1, 64), N=N, K=8 * _log(rng, 8, 2304), bias=rng.random() < 0.7,
                    act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                    residual=rng.random() < 0.5)
    D = rng.choice([64, 96, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([1, 8, 16, 24, 32, 64, 128])
    if op == "rope":
        return dict(op=op, M=_log(rng, 1, 4096), Hq=Hkv * rng.choice([1, 3, 4, 7, 8]), Hkv=Hkv, D=D,
                    rot=rng.choice([16, 32, D // 2, D]), page=page,
                    interleaved=rng.random() < 0.5, hnd=rng.random() < 0.5)
    R = _log(rng, 1, 64)
    most = max(1, min(65536, int(5e8 / (4 * R * Hkv * D))))
    longest = _log(rng, 1, most)
    windowed = rng.random() < 0.4
    return dict(op=op, R=R, Hq=Hkv * rng.choice([1, 2, 4, 5, 7, 8, 12, 16, 32]), Hkv=Hkv, D=D,
                longest=longest, ragged=rng.random() < 0.7, page=page,
                window=_log(rng, 1, 4096) if windowed else 0,
                sinks=rng.choice([0, 1, 4, 16]) if windowed else 0, hnd=rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, mean=0.0):
    """BF16 normals, drawn in pieces of at most 2^27 values so that the 32-bit draws stay small."""
    out = torch.empty(shape, dtype=BF, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV).mul_(std).add_(mean))
    return out


def _cache(g, pages, case, fill=True):
    """A key or value pool as the [pages, page, heads, D] view that both sides take; hnd: the
    memory has each page's tokens of one head side by side."""
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    shape = (pages, Hkv, page, D) if case["hnd"] else (pages, page, Hkv, D)
    t = _randn(g, *shape) if fill else torch.zeros(shape, dtype=BF, device=DEV)
    return t.transpose(1, 2) if case["hnd"] else t


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(case=case, x=_randn(g, M, K), W=_randn(g, N, K, std=K ** -0.5),
                    bias=_randn(g, N, std=0.5) if case["bias"] else None,
                    residual=_randn(g, M, N) if case["residual"] else None,
                    out=torch.empty(M, N, dtype=BF, device=DEV))
    if op == "rope":
        M, Hq, Hkv, D, rot = case["M"], case["Hq"], case["Hkv"], case["D"], case["rot"]
        max_pos = 16384
        # Angles in 64 bits: those of far positions lose their fraction in 32.
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        angle = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * freq
        pages = M // case["page"] + 8
        # Every eighth row or so is padding: computed, but not stored in the cache.
        slots = torch.randperm(pages * case["page"], generator=g, device=DEV)[:M]
        if M > 1:
            slots[torch.rand(M, generator=g, device=DEV) < 0.12] = -1
        kept = torch.nonzero(slots >= 0)[:, 0]
        return dict(case=case, qkv=_randn(g, M, (Hq + 2 * Hkv) * D, std=1.7), kept=kept,
                    q_gamma=_randn(g, D, std=0.1, mean=1.0), k_gamma=_randn(g, D, std=0.1, mean=1.0),
                    rope=torch.cat([angle.cos(), angle.sin()], dim=1).float(),
                    positions=torch.randint(0, max_pos, (M,), generator=g, device=DEV, dtype=torch.int32),
                    slots=slots, k_cache=_cache(g, pages, case), v_cache=_cache(g, pages, case),
                    q_out=torch.empty(M, Hq, D, dtype=BF, device=DEV))
    R, Hq, D, page, longest = case["R"], case["Hq"], case["D"], case["page"], case["longest"]
    lengths = torch.full((R,), longest, dtype=torch.int32, device=DEV)
    if case["ragged"]:
        lengths = torch.randint(1, longest + 1, (R,), generator=g, device=DEV, dtype=torch.int32)
        lengths[0] = longest
        if R > 3:
            lengths[R - 1] = 0  # a padding row of the batch
            lengths[R // 2] = 1
    table_width = -(-longest // page)
    pages = R * table_width
    table = torch.randperm(pages, generator=g, device=DEV).view(R, table_width).to(torch.int32)
    return dict(case=case, q=_randn(g, R, Hq, D, std=1.4), k_cache=_cache(g, pages, case),
                v_cache=_cache(g, pages, case), table=table, lengths=lengths,
                out=torch.empty(R, Hq, D, dtype=BF, device=DEV),
                lse=torch.empty(R, Hq, dtype=torch.float32, device=DEV))


# ---- one pass ------------------------------------------------------------------------

def run(s):
    return {"epilogue": _epilogue, "rope": _rope, "attention": _attention}[s["case"]["op"]](s)


def _epilogue(s):
    act = s["case"]["act"]
    if own:
        import skinny_bf16_gemm_gb300 as sk
        return sk.decode_gemm_bf16_epilogue(s["x"], s["W"], s["out"], bias=s["bias"], activation=act,
                                            residual=s["residual"])
    v = s["x"].float() @ s["W"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    if act == "relu":
        v = torch.where(v > 0, v, torch.zeros_like(v))
    elif act == "silu":
        v = v / (1 + torch.exp(-v))
    elif act == "gelu":
        v = 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        v = 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(BF)


def _norm_rotate(x, gamma, cos, sin, rot, interleaved, eps):
    """x [M, heads, D] in 32 bits: each head's RMSNorm, then its first `rot` values rotated."""
    x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps) * gamma.float()
    y = x.clone()
    c, n = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * c - b * n
        y[..., 1:rot:2] = b * c + a * n
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2] = a * c - b * n
        y[..., rot // 2: rot] = b * c + a * n
    return y


def _rope(s):
    c = s["case"]
    if own:
        import skinny_bf16_gemm_gb300 as sk
        sk.qk_norm_rope_bf16(s["qkv"], c["Hq"], c["Hkv"], s["q_gamma"], s["k_gamma"], s["rope"],
                             s["positions"], s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                             slots=s["slots"], eps=1e-6, interleaved=c["interleaved"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    M, Hq, Hkv, D, rot, page = c["M"], c["Hq"], c["Hkv"], c["D"], c["rot"], c["page"]
    x = s["qkv"].view(M, Hq + 2 * Hkv, D)
    row = s["rope"][s["positions"].long()]
    cos, sin = row[:, : rot // 2], row[:, rot // 2:]
    q = _norm_rotate(x[:, :Hq].float(), s["q_gamma"], cos, sin, rot, c["interleaved"], 1e-6).to(BF)
    k = _norm_rotate(x[:, Hq:Hq + Hkv].float(), s["k_gamma"], cos, sin, rot, c["interleaved"], 1e-6).to(BF)
    slot = s["slots"][s["kept"]]
    s["k_cache"][slot // page, slot % page] = k[s["kept"]]
    s["v_cache"][slot // page, slot % page] = x[:, Hq + Hkv:][s["kept"]]
    return q, s["k_cache"], s["v_cache"]


def _attention(s):
    c = s["case"]
    if own:
        import skinny_bf16_gemm_gb300 as sk
        sk.decode_attention_bf16(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["out"],
                                 window=c["window"], sinks=c["sinks"], lse=s["lse"])
        return s["out"], s["lse"]
    R, Hq, Hkv, D, L = c["R"], c["Hq"], c["Hkv"], c["D"], c["longest"]
    at = s["table"].long()
    k = s["k_cache"][at].reshape(R, -1, Hkv, D)[:, :L].permute(0, 2, 1, 3).float()  # [R, Hkv, L, D]
    v = s["v_cache"][at].reshape(R, -1, Hkv, D)[:, :L].permute(0, 2, 1, 3).float()
    q = s["q"].float().view(R, Hkv, Hq // Hkv, D)
    score = (q @ k.transpose(2, 3)) * D ** -0.5  # [R, Hkv, G, L]
    j = torch.arange(L, device=DEV)[None, :]
    n = s["lengths"].long()[:, None]
    seen = j < n
    if c["window"]:
        seen = seen & ((j >= n - c["window"]) | (j < c["sinks"]))
    seen = seen[:, None, None, :]
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    m = score.max(-1, keepdim=True).values
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(score - m)
    total = p.sum(-1, keepdim=True)
    # A row that sees nothing has a zero output and a log-sum of -inf.
    out = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = m + torch.log(total)
    return out.to(BF).view(R, Hq, D), lse.view(R, Hq)


# ---- what a pass cannot do without -----------------------------------------------------

def _seen(case):
    """Tokens that all rows of an attention case see together (ragged rows at their mean)."""
    R, longest = case["R"], case["longest"]

    def seen(n):
        return n if not case["window"] else min(n, case["window"] + min(case["sinks"], n))

    if not case["ragged"]:
        return R * seen(longest)
    drawn = R - 1 - (2 if R > 3 else 0)
    mean = sum(seen(1 + (2 * i + 1) * longest // 64) for i in range(32)) / 32
    return seen(longest) + drawn * mean


def work(case):
    if case["op"] == "epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * (N * K + M * K + M * N + (N if case["bias"] else 0) + (M * N if case["residual"] else 0)),
                "flops": 2 * M * N * K}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rope":
        M = case["M"]
        return {"bytes": 2 * 2 * M * (Hq + 2 * Hkv) * D + M * (4 * case["rot"] + 12),
                "flops": M * (Hq + Hkv) * (4 * D + 3 * case["rot"])}
    n = _seen(case)
    return {"bytes": 4 * n * Hkv * D + 4 * n / case["page"] + 4 * case["R"] * Hq * D + 4 * case["R"] * (Hq + 1),
            "flops": 4 * n * Hq * D}


# ---- 64 bits -------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "epilogue":
        v = torch.einsum("mk,nk->mn", s["x"].to(f64), s["W"].to(f64))
        if s["bias"] is not None:
            v += s["bias"].to(f64)
        act = case["act"]
        if act == "relu":
            v = v.clamp(min=0)
        elif act == "silu":
            v = v * torch.sigmoid(v)
        elif act == "gelu":
            v = v * torch.special.ndtr(v)
        elif act == "gelu_tanh":
            v = v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
        return v + s["residual"].to(f64) if s["residual"] is not None else v
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "rope":
        M, rot = case["M"], case["rot"]
        k64, v64 = s["k_cache"].to(f64), s["v_cache"].to(f64)
        rows = s["qkv"].to(f64).view(M, Hq + 2 * Hkv, D)
        turn = s["rope"].to(f64)[s["positions"].long()]
        turn = torch.complex(turn[:, : rot // 2], turn[:, rot // 2:])[:, None, :]

        def head(x, gamma):
            x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * gamma.to(f64)
            first = x[..., :rot]
            pair = first.unflatten(-1, (-1, 2)) if case["interleaved"] else first.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_real(torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * turn)
            z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return torch.cat([z, x[..., rot:]], -1)

        q, k = head(rows[:, :Hq], s["q_gamma"]), head(rows[:, Hq:Hq + Hkv], s["k_gamma"])
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                k64[slot // page, slot % page] = k[i]
                v64[slot // page, slot % page] = rows[i, Hq + Hkv:]
        return q, k64, v64
    R, G = case["R"], Hq // Hkv
    out = torch.zeros(R, Hq, D, dtype=f64, device=DEV)
    lse = torch.full((R, Hq), -math.inf, dtype=f64, device=DEV)
    for r, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        seen = torch.arange(n, device=DEV)
        if case["window"]:
            seen = seen[(seen >= n - case["window"]) | (seen < case["sinks"])]
        at, off = s["table"][r].long()[seen // page], seen % page
        for h in range(Hkv):
            k, v = s["k_cache"][at, off, h].to(f64), s["v_cache"][at, off, h].to(f64)
            score = s["q"][r, h * G:(h + 1) * G].to(f64) @ k.t() / math.sqrt(D)
            lse[r, h * G:(h + 1) * G] = torch.logsumexp(score, -1)
            out[r, h * G:(h + 1) * G] = torch.softmax(score, -1) @ v
    return out, lse
