"""The operators of a decode step that serves many requests, as measured cases.

  logprobs  token_logprobs_bf16: log probabilities of given tokens, the entropy and the
            top alternatives of every row of logits
  lora      decode_gemm_bf16_lora: out = act(x W^T + c_a (x A_a^T) B_a^T + bias) + residual,
            each row with an adapter a of its own, or none
  prefix    decode_attention_shared_prefix_bf16: one new token per row over a prefix that all
            rows share and the row's own tokens, both in a paged cache

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
        # One drafted token over one rank's vocabulary shard: latency.
        dict(name="logprobs 1x20480 top 1", op="logprobs", M=1, V=20480, T=1, top=1, masked=False),
        # A ragged batch over a vocabulary of odd size: rows that start anywhere.
        dict(name="logprobs 17x50257 top 5", op="logprobs", M=17, V=50257, T=1, top=5, masked=False),
        # A full decode batch over the whole vocabulary (eight shards), part of it forbidden by a
        # grammar, several candidates asked for, and the alternatives that a client may ask for.
        dict(name="logprobs 64x163840 top 20", op="logprobs", M=64, V=163840, T=4, top=20, masked=True),
        # A prompt's tokens scored.
        dict(name="logprobs 2048x163840 top 8", op="logprobs", M=2048, V=163840, T=1, top=8, masked=False),
        # One request with its adapter through a small projection: latency.
        dict(name="lora 1x2048x7168 rank 16", op="lora", M=1, N=2048, K=7168, E=8, rank=16, act="silu",
             bias=True, residual=False),
        # Ragged everything: odd rows, an odd output width, K that ends inside a block.
        dict(name="lora 5x4099x1000 rank 8", op="lora", M=5, N=4099, K=1000, E=3, rank=8, act="relu",
             bias=True, residual=True),
        # The up linear of 16 requests with their activation, large adapters.
        dict(name="lora 16x18432x7168 rank 64", op="lora", M=16, N=18432, K=7168, E=16, rank=64,
             act="gelu_tanh", bias=True, residual=False),
        # The down linear of a full batch, an adapter for nearly every request.
        dict(name="lora 64x7168x18432 rank 16", op="lora", M=64, N=7168, K=18432, E=64, rank=16, act="none",
             bias=False, residual=True),
        # A few requests behind a short common prompt, one tensor-parallel rank's heads: latency.
        dict(name="prefix 4 rows 509 + 64", op="prefix", R=4, Hq=7, Hkv=1, D=128, prefix=509, longest=64,
             page=16, hnd=False),
        # A full batch of one rank behind a long system prompt, answers of up to 1000 tokens.
        dict(name="prefix 64 rows 16001 + 1000", op="prefix", R=64, Hq=7, Hkv=1, D=128, prefix=16001,
             longest=1000, page=16, hnd=False),
        # Small heads in groups of four, pages by head.
        dict(name="prefix 32 rows 32768 + 2000", op="prefix", R=32, Hq=32, Hkv=8, D=64, prefix=32768,
             longest=2000, page=64, hnd=True),
        # A full batch that asks about one long document, all heads on one GPU.
        dict(name="prefix 64 rows 65521 + 1000", op="prefix", R=64, Hq=56, Hkv=8, D=128, prefix=65521,
             longest=1000, page=32, hnd=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "lora", "prefix"])
    if op == "logprobs":
        V = _log(rng, 100, 200000)
        return dict(op=op, M=_log(rng, 1, min(4096, 2048 * 163840 // V)), V=V, T=rng.choice([1, 1, 2, 5]),
                    top=rng.choice([0, 1, 2, 5, 8, 20, 32]), masked=rng.random() < 0.3)
    if op == "lora":
        rank = rng.choice([8, 16, 24, 32, 64, 128])
        return dict(op=op, M=rng.randint(1, 64), N=_log(rng, 100, 20480), K=8 * _log(rng, 8, 2304),
                    E=rng.randint(1, min(64, 2048 // rank)), rank=rank,
                    act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), bias=rng.random() < 0.6,
                    residual=rng.random() < 0.5)
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 192, 256])
    R, Hq = _log(rng, 1, 128), Hkv * rng.choice([1, 3, 4, 7, 8, 12, 16])
    return dict(op=op, R=R, Hq=Hq, Hkv=Hkv, D=D,
                prefix=_log(rng, 1, max(1, min(65536, int(2.5e10 / (R * Hq * D))))),
                longest=_log(rng, 1, max(1, min(4096, int(2e8 / (4 * R * Hkv * D))))),
                page=rng.choice([1, 8, 16, 24, 32, 64, 128]), hnd=rng.random() < 0.5)


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


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "logprobs":
        M, V, T, top = case["M"], case["V"], case["T"], case["top"]
        logits = _randn(g, M, V, std=2.5)
        tokens = torch.randint(0, V, (M, T), generator=g, device=DEV)
        # The tokens asked for are likely ones, some of them far above the rest.
        lift = 3 + 9 * torch.rand(M, 1, generator=g, device=DEV)
        logits.scatter_(1, tokens, (logits.gather(1, tokens).float() + lift).to(BF))
        if case["masked"]:  # forbidden tokens
            for r in range(0, M, 2):
                logits[r, torch.rand(V, generator=g, device=DEV) < 0.9] = -math.inf
            logits.scatter_(1, tokens[:, :1], 4.0)
        if M > 3:
            tokens[M // 3] = -1  # a position that is not asked for
        return dict(case=case, logits=logits, tokens=tokens,
                    logprobs=torch.empty(M, T, dtype=torch.float32, device=DEV),
                    entropy=torch.empty(M, dtype=torch.float32, device=DEV),
                    top_logprobs=torch.empty(M, top, dtype=torch.float32, device=DEV) if top else None,
                    top_tokens=torch.empty(M, top, dtype=torch.int64, device=DEV) if top else None)
    if op == "lora":
        M, N, K, E, rank = case["M"], case["N"], case["K"], case["E"], case["rank"]
        # As many different adapters as there are, dealt to the rows in any order.
        adapters = (torch.randperm(M, generator=g, device=DEV) % E).to(torch.int32)
        if M > 2:
            adapters[torch.rand(M, generator=g, device=DEV) < 0.1] = -1  # requests without one
        return dict(case=case, x=_randn(g, M, K), W=_randn(g, N, K, std=K ** -0.5),
                    A=_randn(g, E, rank, K, std=K ** -0.5), B=_randn(g, E, N, rank, std=rank ** -0.5),
                    adapters=adapters, scales=0.25 + torch.rand(E, generator=g, device=DEV),
                    bias=_randn(g, N, std=0.5) if case["bias"] else None,
                    residual=_randn(g, M, N) if case["residual"] else None,
                    out=torch.empty(M, N, dtype=BF, device=DEV))
    R, Hq, Hkv, D, page = case["R"], case["Hq"], case["Hkv"], case["D"], case["page"]
    lengths = torch.randint(1, case["longest"] + 1, (R,), generator=g, device=DEV, dtype=torch.int32)
    lengths[0] = case["longest"]
    if R > 3:
        lengths[R - 1] = 0  # a row with the prefix alone
        lengths[R // 2] = 1
    width, shared = -(-case["longest"] // page), -(-case["prefix"] // page)
    pages = shared + R * width
    place = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    shape = (pages, Hkv, page, D) if case["hnd"] else (pages, page, Hkv, D)
    k, v = _randn(g, *shape), _randn(g, *shape)
    # Keys and values as [pages, page, heads, D] views; hnd: each page's tokens of one head side by side.
    return dict(case=case, q=_randn(g, R, Hq, D, std=1.4), k_cache=k.transpose(1, 2) if case["hnd"] else k,
                v_cache=v.transpose(1, 2) if case["hnd"] else v, prefix_table=place[:shared].clone(),
                prefix_length=torch.full((1,), case["prefix"], dtype=torch.int32, device=DEV),
                table=place[shared:].view(R, width).clone(), lengths=lengths,
                out=torch.empty(R, Hq, D, dtype=BF, device=DEV),
                lse=torch.empty(R, Hq, dtype=torch.float32, device=DEV))


# ---- one pass ------------------------------------------------------------------------

def run(s):
    return {"logprobs": _logprobs, "lora": _lora, "prefix": _prefix}[s["case"]["op"]](s)


def _logprobs(s):
    c = s["case"]
    if own:
        import skinny_bf16_gemm_gb300 as sk
        sk.token_logprobs_bf16(s["logits"], s["tokens"], s["logprobs"], entropy=s["entropy"],
                               top_logprobs=s["top_logprobs"], top_tokens=s["top_tokens"])
        return s["logprobs"], s["entropy"], s["top_logprobs"], s["top_tokens"]
    x = s["logits"].float()
    x = x - x.max(-1, keepdim=True).values
    e = torch.exp(x)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    # Forbidden tokens (-inf) add nothing to the entropy.
    xe = torch.where(e > 0, x * e, torch.zeros_like(x)).sum(-1)
    entropy = log_total[:, 0] - xe / total[:, 0]
    given = torch.gather(x, 1, s["tokens"].clamp(min=0)) - log_total
    given = torch.where(s["tokens"] >= 0, given, torch.zeros_like(given))
    if not c["top"]:
        return given, entropy, None, None
    order = torch.sort(x, dim=-1, descending=True, stable=True)
    return (given, entropy, order.values[:, :c["top"]] - log_total,
            order.indices[:, :c["top"]].contiguous())


def _lora(s):
    act = s["case"]["act"]
    if own:
        import skinny_bf16_gemm_gb300 as sk
        return sk.decode_gemm_bf16_lora(s["x"], s["W"], s["out"], s["A"], s["B"], s["adapters"],
                                        scales=s["scales"], bias=s["bias"], activation=act,
                                        residual=s["residual"])
    x = s["x"].float()
    v = x @ s["W"].float().t()
    a = s["adapters"].long()
    at = a.clamp(min=0)
    t = (s["A"][at].float() @ x[:, :, None])[:, :, 0] * (s["scales"][at] * (a >= 0))[:, None]  # [M, rank]
    v = v + (s["B"][at].float() @ t[:, :, None])[:, :, 0]
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


def _prefix(s):
    c = s["case"]
    if own:
        import skinny_bf16_gemm_gb300 as sk
        sk.decode_attention_shared_prefix_bf16(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"],
                                               s["prefix_length"], s["table"], s["lengths"], s["out"],
                                               lse=s["lse"])
        return s["out"], s["lse"]
    R, Hq, Hkv, D, P, L = c["R"], c["Hq"], c["Hkv"], c["D"], c["prefix"], c["longest"]
    G = Hq // Hkv
    at, mine = s["prefix_table"].long(), s["table"].long()
    kp = s["k_cache"][at].reshape(-1, Hkv, D)[:P].permute(1, 0, 2).float()  # [Hkv, P, D]
    vp = s["v_cache"][at].reshape(-1, Hkv, D)[:P].permute(1, 0, 2).float()
    ko = s["k_cache"][mine].reshape(R, -1, Hkv, D)[:, :L].permute(0, 2, 1, 3).float()  # [R, Hkv, L, D]
    vo = s["v_cache"][mine].reshape(R, -1, Hkv, D)[:, :L].permute(0, 2, 1, 3).float()
    q = s["q"].float().view(R, Hkv, G, D)
    q_all = q.permute(1, 0, 2, 3).reshape(Hkv, R * G, D)
    shared = (q_all @ kp.transpose(1, 2)) * D ** -0.5  # [Hkv, R * G, P]
    score = (q @ ko.transpose(2, 3)) * D ** -0.5  # [R, Hkv, G, L]
    seen = (torch.arange(L, device=DEV)[None, :] < s["lengths"].long()[:, None])[:, None, None, :]
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    # The prefix is never empty: the maximum is finite.
    mp = shared.max(-1, keepdim=True).values.view(Hkv, R, G, 1).permute(1, 0, 2, 3)
    m = torch.maximum(score.max(-1, keepdim=True).values, mp)  # [R, Hkv, G, 1]
    ps = torch.exp(shared - m.permute(1, 0, 2, 3).reshape(Hkv, R * G, 1))
    po = torch.exp(score - m)
    total = po.sum(-1, keepdim=True) + ps.sum(-1).view(Hkv, R, G, 1).permute(1, 0, 2, 3)
    out = (po @ vo + (ps @ vp).view(Hkv, R, G, D).permute(1, 0, 2, 3)) / total
    return out.reshape(R, Hq, D).to(BF), (m + torch.log(total)).reshape(R, Hq)


# ---- what a pass cannot do without -----------------------------------------------------

def work(case):
    if case["op"] == "logprobs":
        M, V = case["M"], case["V"]
        return {"bytes": M * (2 * V + 12 * case["T"] + 4 + 12 * case["top"]), "flops": 5 * M * V}
    if case["op"] == "lora":
        M, N, K, rank = case["M"], case["N"], case["K"], case["rank"]
        used = min(M, case["E"])
        return {"bytes": 2 * (N * K + M * K + M * N + (N if case["bias"] else 0) +
                              (M * N if case["residual"] else 0) + used * rank * (N + K)) + 4 * (M + used),
                "flops": 2 * M * N * K + 2 * M * rank * (N + K)}
    R, Hq, Hkv, D = case["R"], case["Hq"], case["Hkv"], case["D"]
    mean = case["longest"] * (1 if R == 1 else 0.5)  # of the rows' own tokens
    tokens = case["prefix"] + R * mean
    return {"bytes": int(4 * tokens * Hkv * D + 4 * tokens / case["page"] + 4 * R * Hq * D + 4 * R * (Hq + 1)),
            "flops": int(4 * Hq * D * R * (case["prefix"] + mean))}


# ---- 64 bits -------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "logprobs":
        lps, ents, tops, ids = [], [], [], []
        V, top = case["V"], case["top"]
        back = (1 << 32) - 1 - torch.arange(V, device=DEV)  # of equal logits the lower index first
        for r0 in range(0, case["M"], 64):
            bits = s["logits"][r0:r0 + 64]
            lp = torch.log_softmax(bits.to(f64), -1)
            ents.append(torch.special.entr(lp.exp()).sum(-1))
            t = s["tokens"][r0:r0 + 64]
            rows = torch.arange(t.shape[0], device=DEV)[:, None]
            lps.append(lp[rows, t.clamp(min=0)].masked_fill(t < 0, 0.0))
            if top:
                # A whole number for every logit, in the logits' order and no two alike.
                b = bits.view(torch.int16).long()
                key = torch.where(b < 0, -(b & 0x7FFF), b) * (1 << 32) + back
                i = torch.topk(key, top, dim=-1).indices
                ids.append(i)
                tops.append(lp[rows, i])
        return torch.cat(lps), torch.cat(ents), torch.cat(tops) if top else None, torch.cat(ids) if top else None
    if case["op"] == "lora":
        x = s["x"].to(f64)
        v = torch.einsum("mk,nk->mn", x, s["W"].to(f64))
        for m, a in enumerate(s["adapters"].tolist()):
            if a >= 0:
                v[m] += s["scales"][a].to(f64) * (s["B"][a].to(f64) @ (s["A"][a].to(f64) @ x[m]))
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
    R, Hq, Hkv, D, page = case["R"], case["Hq"], case["Hkv"], case["D"], case["page"]
    G = Hq // Hkv
    out = torch.zeros(R, Hq, D, dtype=f64, device=DEV)
    lse = torch.zeros(R, Hq, dtype=f64, device=DEV)
    j = torch.arange(case["prefix"], device=DEV)
    at, off = s["prefix_table"].long()[j // page], j % page
    kp, vp = s["k_cache"][at, off].to(f64), s["v_cache"][at, off].to(f64)  # [P, Hkv, D]
    for r, n in enumerate(s["lengths"].tolist()):
        j = torch.arange(n, device=DEV)
        at, off = s["table"][r].long()[j // page], j % page
        for h in range(Hkv):
            k = torch.cat([kp[:, h], s["k_cache"][at, off, h].to(f64)])
            v = torch.cat([vp[:, h], s["v_cache"][at, off, h].to(f64)])
            score = s["q"][r, h * G:(h + 1) * G].to(f64) @ k.t() / math.sqrt(D)
            lse[r, h * G:(h + 1) * G] = torch.logsumexp(score, -1)
            out[r, h * G:(h + 1) * G] = torch.softmax(score, -1) @ v
    return out, lse
