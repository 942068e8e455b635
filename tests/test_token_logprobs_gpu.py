"""token_logprobs_bf16 against a plain implementation in 64 bits, at the sizes, ties, masks
and alignments where it can go wrong."""
import math

import pytest
import torch

import skinny_bf16_gemm_gb300 as sk

pytestmark = pytest.mark.gpu
F64 = torch.float64
U32 = 2.0 ** -24  # half an FP32 step, relative


def reference(x, tokens, top):
    """(logprobs, entropy, lse, top logprobs, top tokens) in 64 bits, and their tolerances.

    A weight exp(t), t = x - m <= 0, is off by t's rounding U32 |t|, its product with log2 e
    U32 |t|, and the exponential's 2 ulp, 2^-22; the sum of V weights takes at most n =
    V / 256 + 80 additions one after another (a thread's own, with rescaling, then joins; one
    CTA of 128 threads a row, V / 128 + 15, is for no V here where that is more).
    So S is off by ds = 2^-22 + 2 U32 E|t| + 2 n U32 relative, E the mean over p, and the
    sum of p t by E|t| (2^-22 + 3 U32 + 2 n U32) + 2 U32 E t^2; logarithm, quotient and
    differences by 4 U32 of their results and terms."""
    x = x.to(F64)
    V = x.shape[1]
    m = x.amax(1, keepdim=True)
    t = x - m
    e = t.exp()
    S = e.sum(1, keepdim=True)
    p = e / S
    t0 = torch.where(p > 0, t, torch.zeros_like(t))
    e1, e2 = (p * t0).sum(1), (p * t0 * t0).sum(1)
    n = V / 256 + 80
    ds = 2.0 ** -22 - 2 * U32 * e1 + 2 * n * U32
    logS = S.log()[:, 0]
    lse = m[:, 0] + logS
    lse_tol = ds + 4 * U32 * (lse.abs() + m[:, 0].abs() + logS)
    ent = logS - e1
    ent_tol = ds - e1 * (2.0 ** -22 + 3 * U32 + 2 * n * U32 + ds) + 2 * U32 * e2 + 4 * U32 * (ent.abs() + logS - e1)
    lp = t - logS[:, None]
    lp_tol = ds[:, None] + 4 * U32 * (t.abs() + logS[:, None])
    lp_tol = torch.where(torch.isfinite(lp), lp_tol, torch.zeros_like(lp))
    at = tokens.clamp(min=0)
    given = torch.where(tokens >= 0, lp.gather(1, at), torch.zeros_like(at, dtype=F64))
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    return dict(logprobs=(given, lp_tol.gather(1, at)), entropy=(ent, ent_tol), lse=(lse, lse_tol),
                top_logprobs=(lp.gather(1, order), lp_tol.gather(1, order))), order


def call(x, tokens, top, **kw):
    M, T = tokens.shape
    new = lambda *s, dtype=torch.float32: torch.full(s, 77, dtype=dtype, device="cuda")  # noqa: E731
    out = dict(logprobs=new(M, T), entropy=new(M), lse=new(M))
    if top:
        out.update(top_logprobs=new(M, top), top_tokens=new(M, top, dtype=torch.int64))
    got = sk.token_logprobs_bf16(x, tokens, **out, **kw)
    assert got is out["logprobs"]
    return out


def check(x, tokens, top, **kw):
    got = call(x, tokens, top, **kw)
    want, order = reference(x, tokens, top)
    for name, (w, tol) in want.items():
        if name not in got:
            continue
        g = got[name].to(F64)
        fine = torch.isfinite(w)
        assert torch.equal(g[~fine], w[~fine]), name
        over = ((g - w).abs() - tol)[fine]
        assert over.numel() == 0 or over.max() <= 0, (name, over.max().item())
    if top:
        assert torch.equal(got["top_tokens"], order)
    assert sk.device_error()[0] == 0
    return got


def logits(M, V, seed, std=2.5, offset=0, pad=0):
    """Rows of V logits, `offset` values into a row of V + offset + pad."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(M, V + offset + pad, generator=g, device="cuda") * std
    return x.to(torch.bfloat16)[:, offset:offset + V]


def some_tokens(M, V, T, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(0, V, (M, T), generator=g, device="cuda")


# One value, less than a vector, less than a vector a thread, each cluster size on both
# sides of its rule, several rounds of a thread; odd rows at every alignment.
@pytest.mark.parametrize("M,V,top", [(1, 1, 1), (3, 2, 2), (2, 7, 7), (5, 8, 8), (4, 33, 32), (2, 255, 20),
                                     (3, 2047, 20), (1, 2049, 1), (2, 4096, 32), (1, 8191, 20),
                                     (1, 16384, 32), (1, 16400, 5), (7, 20480, 20), (64, 50257, 5),
                                     (160, 20000, 8), (400, 10001, 32), (1300, 3000, 4), (2, 163840, 32),
                                     (1600, 80008, 8), (3000, 9, 3), (900, 700, 32)])
def test_sizes(cuda_ok, M, V, top):
    check(logits(M, V, seed=V), some_tokens(M, V, 3, seed=M), top)


@pytest.mark.parametrize("offset", range(8))
def test_rows_at_any_alignment(cuda_ok, offset):
    for V in (5, 4099, 30001):
        check(logits(4, V, seed=offset, offset=offset, pad=3), some_tokens(4, V, 1, seed=V), 20 if V > 20 else 3)


def test_values_around_a_row_are_not_read(cuda_ok):
    buf = torch.full((6, 3016), math.inf, dtype=torch.bfloat16, device="cuda")
    x = buf[:, 5:3005]
    x.copy_(logits(6, 3000, seed=3))
    check(x, some_tokens(6, 3000, 2, seed=4), 20)


# Many equal values: all equal; a few levels; ties that fill a whole list and begin late.
def test_ties_go_to_the_lowest_index(cuda_ok):
    tokens = some_tokens(3, 40000, 1, seed=1)
    check(torch.zeros(3, 40000, dtype=torch.bfloat16, device="cuda"), tokens, 32)
    x = logits(3, 40000, seed=2)
    check((x.float() / 2).round().to(torch.bfloat16), tokens, 32)
    late = torch.full((3, 40000), -4.0, dtype=torch.bfloat16, device="cuda")
    late[:, 39000:] = 1.0
    late[1, 39990:] = 2.0
    late[2, 7] = 1.0
    check(late, tokens, 32)
    signs = torch.zeros(3, 40000, dtype=torch.bfloat16, device="cuda")
    signs[:, ::2] = -0.0
    check(signs, tokens, 20)


# A thread's values all large: every value of few threads is over the bound.
@pytest.mark.parametrize("V", [16384, 163840])
def test_large_values_in_few_threads(cuda_ok, V):
    for rows in (1, 300):
        x = logits(rows, V, seed=5, std=0.5)
        n = 8 * 256  # values of one round of a CTA's threads
        for r in range(0, rows, 37):
            for lane in range(31):
                for e in range(8):
                    x[r, lane * 8 + e::n] = 20 + (lane + e) % 3
        check(x, some_tokens(rows, V, 1, seed=6), 32)


@pytest.mark.parametrize("fill", [-math.inf, torch.finfo(torch.bfloat16).min])
def test_masked_values(cuda_ok, fill):
    x = logits(6, 20481, seed=7)
    keep = torch.zeros_like(x, dtype=torch.bool)
    keep[0, 20480] = True  # a single one left, the last
    keep[1, 0] = True
    keep[2, 100:103] = True
    keep[3, ::7] = True
    keep[4] = True
    keep[5, 5000:5600] = True
    x = torch.where(keep, x, torch.full_like(x, fill))
    tokens = torch.tensor([[20480, 3], [0, 1], [101, 102], [7, 14], [1, 2], [5001, 0]], device="cuda")
    got = check(x, tokens, 20)
    assert got["entropy"][0] == 0 and got["logprobs"][0, 0] == 0


def test_rows_that_have_no_probabilities(cuda_ok):
    x = logits(5, 9000, seed=8)
    clean = x.clone()
    x[1] = -math.inf
    x[2, 4000] = math.nan
    x[3, 17] = math.inf
    tokens = some_tokens(5, 9000, 2, seed=9)
    got = call(x, tokens, 5)
    for r in (2, 3):
        assert torch.isnan(got["lse"][r]) and torch.isnan(got["entropy"][r])
        assert torch.isnan(got["logprobs"][r]).all() and torch.isnan(got["top_logprobs"][r]).all()
    assert got["lse"][1] == -math.inf and torch.isnan(got["entropy"][1])
    assert torch.isnan(got["logprobs"][1]).all()
    assert got["top_tokens"][1].tolist() == [0, 1, 2, 3, 4] and got["top_tokens"][3, 0] == 17
    x2 = x.clone()
    x2[2, 4000] = -math.inf  # in the order of values NaN is -inf
    assert torch.equal(got["top_tokens"][2], torch.sort(x2[2].double(), descending=True, stable=True).indices[:5])
    alone = call(clean, tokens, 5)
    for name in got:  # the other rows as without them
        assert torch.equal(got[name][[0, 4]], alone[name][[0, 4]]), name


def test_tokens_not_asked_for_and_out_of_range(cuda_ok):
    x = logits(4, 3001, seed=10)
    tokens = torch.tensor([[-1, 5], [3000, -100], [2, 2], [3001, 0]], device="cuda")
    got = call(x, tokens, 0)
    assert got["logprobs"][0, 0] == 0 and got["logprobs"][1, 1] == 0
    assert torch.isnan(got["logprobs"][3, 0]) and torch.isfinite(got["logprobs"][3, 1])
    st, word = sk.device_error()
    assert sk.STATUS[st] == "SKINNY_ERR_INDEX" and word == 256
    assert sk.device_error() == (0, 0)


def test_optional_results(cuda_ok):
    x = logits(9, 5000, seed=11)
    tokens = some_tokens(9, 5000, 1, seed=12)
    full = check(x, tokens, 6)
    one = torch.empty(9, device="cuda")
    sk.token_logprobs_bf16(x, tokens[:, 0].contiguous(), one)
    assert torch.equal(one, full["logprobs"][:, 0])
    ent, ids = torch.empty(9, device="cuda"), torch.empty(9, 6, dtype=torch.int64, device="cuda")
    assert sk.token_logprobs_bf16(x, None, None, entropy=ent, top_tokens=ids) is None
    assert torch.equal(ent, full["entropy"]) and torch.equal(ids, full["top_tokens"])
    tlp = torch.empty(9, 6, device="cuda")
    sk.token_logprobs_bf16(x, None, None, top_logprobs=tlp, pdl=True)
    assert torch.equal(tlp, full["top_logprobs"])


def test_captured_and_on_another_stream(cuda_ok):
    x = logits(12, 20480, seed=13)
    tokens = some_tokens(12, 20480, 2, seed=14)
    want = call(x, tokens, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(x, tokens, 8, stream=s)
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call(x, tokens, 8)
    x.copy_(logits(12, 20480, seed=15))
    for _ in range(2):
        g.replay()
    want = call(x, tokens, 8)
    for name in want:
        assert torch.equal(got[name], want[name])


def test_behind_the_lm_head(cuda_ok):
    """The log probabilities of a verification step: the lm_head's logits, the drafted tokens."""
    g = torch.Generator(device="cuda")
    g.manual_seed(16)
    x = torch.randn(8, 512, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(20480, 512, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    out = torch.empty(8, 20000, dtype=torch.bfloat16, device="cuda")
    sk.decode_gemm_bf16_logits(x, W, out, soft_cap=30.0)
    check(out, some_tokens(8, 20000, 1, seed=17), 20)
