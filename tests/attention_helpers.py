"""64-bit references of the attention operators, and the error their kernels may make."""
import math

import torch

F64 = torch.float64
HALF_BF16 = 2.0 ** -8   # half a BF16 step, relative
U32 = 2.0 ** -24        # half an FP32 step, relative


def make_cache(pages, page, heads, D, layout, seed, device="cuda"):
    """(k, v) views [pages, page, heads, D]: 'nhd', 'hnd', 'kv' (keys and values of a page
    side by side in one buffer) or 'padded' (every axis padded by a multiple of 8)."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=device).to(torch.bfloat16)
    if layout == "nhd":
        return rand(pages, page, heads, D), rand(pages, page, heads, D)
    if layout == "hnd":
        return rand(pages, heads, page, D).transpose(1, 2), rand(pages, heads, page, D).transpose(1, 2)
    if layout == "kv":
        kv = rand(pages, 2, page, heads, D)
        return kv[:, 0], kv[:, 1]
    k, v = rand(pages + 1, page + 1, heads + 1, D + 8), rand(pages + 1, page + 1, heads + 1, D + 8)
    return k[1:, :page, 1:, 8:], v[1:, :page, 1:, 8:]


def seen_tokens(n, window, sinks):
    j = torch.arange(n)
    return j if not window else j[(j >= n - window) | (j < sinks)]


def attention_reference(q, k_cache, v_cache, table, lengths, scale, window=0, sinks=0):
    """(out, lse, out_tol, lse_tol) in 64 bits. The tolerances bound the kernel's error:

    scores: FP32 sums of D products, relative to sum |q k| (2 U32 a step allows for an
    accumulation that truncates): ds = 2 (D + 2) U32 max_j sum_i |q_i k_ji| scale, plus
    the scaling's and the exponent's own roundings, 4 U32 |s|;
    weights: exp's relative error ds + 2^-21 (the exponential instruction is 2 ulp); the
    two-term split: truncation leaves less than a step, 2^-7 p, whose rounding is off by
    at most half a step of its own, 2^-8 of it, so 2^-15 p; the weighted mean moves by at
    most twice that times max |v|;
    sums over n tokens in steps of 16, then 4 warps and at most 320 partials, 2 U32 each;
    output: half a BF16 step."""
    R, Hq, D = q.shape
    Hkv, page = k_cache.shape[2], k_cache.shape[1]
    G = Hq // Hkv
    out = torch.zeros(R, Hq, D, dtype=F64, device=q.device)
    lse = torch.full((R, Hq), -math.inf, dtype=F64, device=q.device)
    out_tol = torch.zeros_like(out)
    lse_tol = torch.zeros_like(lse)
    for r, n in enumerate(lengths.tolist()):
        if n == 0:
            continue
        j = seen_tokens(n, window, sinks).to(q.device)
        at, off = table[r].long()[j // page], j % page
        k, v = k_cache[at, off].to(F64), v_cache[at, off].to(F64)  # [n, Hkv, D]
        qr = q[r].to(F64).view(Hkv, G, D)
        s = torch.einsum("hgd,nhd->hgn", qr, k) * scale
        mag = torch.einsum("hgd,nhd->hgn", qr.abs(), k.abs()) * abs(scale)
        ds = 2 * (D + 2) * U32 * mag.amax(-1) + 4 * U32 * s.abs().amax(-1) + 2.0 ** -21
        steps = 2 * U32 * (j.numel() / 16 + 324)
        out[r] = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), v).reshape(Hq, D)
        lse[r] = torch.logsumexp(s, -1).reshape(Hq)
        vmax = v.abs().amax(0)[:, None, :]  # [Hkv, 1, D]
        out_tol[r] = (2 * (ds[..., None] + 2.0 ** -15 + steps) * vmax).expand(Hkv, G, D).reshape(Hq, D)
        out_tol[r] += HALF_BF16 * (out[r].abs() + out_tol[r])
        lse_tol[r] = (ds + steps).reshape(Hq) + 4 * U32 * (1 + lse[r].abs())
    return out, lse, out_tol, lse_tol


def check_close(got, want, tol, name):
    got = got.to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), f"{name}: finite values differ"
    assert torch.equal(got[~fine], want[~fine]), f"{name}: infinities differ"
    over = ((got - want).abs() - tol)[fine]
    if over.numel():
        i = int(over.argmax())
        assert over[i] <= 0, (f"{name}: {got[fine][i].item()} against {want[fine][i].item()}, "
                              f"allowed {tol[fine][i].item()}")


def rope_table(max_pos, rot, device="cuda"):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=F64, device=device) / rot)
    angle = torch.arange(max_pos, dtype=F64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def norm_rope_reference(x, gamma, rope, positions, interleaved, eps):
    """(y, tol) of heads x [M, H, D] in 64 bits. The norm and the two products of a pair
    take fewer than D + 16 FP32 roundings relative to |a| + |b|; then half a BF16 step."""
    x = x.to(F64)
    D = x.shape[-1]
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.to(F64)
    y, mag = x.clone(), x.abs()
    if rope is not None:
        rot = rope.shape[1]
        row = rope.to(F64)[positions.long()][:, None, :]
        c, s = row[..., : rot // 2], row[..., rot // 2:]
        ia = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        ib = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag = mag.clone()
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    tol = (D + 16) * U32 * mag
    return y, tol + HALF_BF16 * (y.abs() + tol)
