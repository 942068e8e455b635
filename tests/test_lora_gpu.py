"""decode_gemm_bf16_lora on the GPU.

Integer inputs (A of -1, 0, 1 with few nonzeros, so that every sum is a whole number below
2^24) without a curved activation are exact in FP32 whatever the order and must match bit for
bit. Otherwise against 64 bits, as for the GEMM's epilogue: an FP32 sum of K products is off by
e = (K / 16 + 48) 2^-23 sum |x w| (up to 32 slices are joined); A x so by da, the scale and the
product with B by 2^-23 (rank + 4) sum |t b| + sum da |b|; adding both 2^-23 of either."""
import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
import workloads
from attention_helpers import F64, HALF_BF16, check_close
from gpu_helpers import Guarded, gemm_inputs_device
from test_epilogue_gpu import activate, extras

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def adapter_ids(M, E, kind, seed):
    """Row by row: 'own' (all different as far as E goes, in any order), 'one', 'pairs', 'none',
    'some' (every third without), 'last' (only the last row has one)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    m = torch.arange(M, device="cuda")
    ids = {"own": torch.randperm(M, generator=g, device="cuda") % E, "one": torch.full_like(m, E - 1),
           "pairs": (m // 2) % E, "none": torch.full_like(m, -1), "some": torch.where(m % 3 == 1, -1, m % E),
           "last": torch.where(m == M - 1, E // 2, -7)}[kind]
    return ids.to(torch.int32)


def pool(E, rank, N, K, seed, kind="normal"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if kind == "int":
        A = torch.zeros(E, rank, K, device="cuda")
        for _ in range(4):  # four nonzeros a row, or fewer
            A.scatter_(2, torch.randint(0, K, (E, rank, 1), generator=g, device="cuda"), 1.0)
        A *= torch.randint(0, 2, (E, rank, 1), generator=g, device="cuda") * 2 - 1
        B = torch.randint(-3, 4, (E, N, rank), generator=g, device="cuda")
        return A.to(BF), B.to(BF), torch.randint(1, 3, (E,), generator=g, device="cuda").float()
    A = torch.randn(E, rank, K, generator=g, device="cuda") * K ** -0.5
    B = torch.randn(E, N, rank, generator=g, device="cuda") * rank ** -0.5
    return A.to(BF), B.to(BF), 0.2 + torch.rand(E, generator=g, device="cuda")


def run(x, W, A, B, ids, scales=None, bias=None, act="none", residual=None, in_place=False, **kw):
    M, N = x.shape[0], W.shape[0]
    out = Guarded((M, N), fill=residual if in_place else None)
    got = sk.decode_gemm_bf16_lora(x, W, out.tensor, A, B, ids, scales, bias, act,
                                   out.tensor if in_place else residual, **kw)
    assert got is out.tensor
    torch.cuda.synchronize()
    out.check()
    assert sk.device_error() == (0, 0)
    return out.tensor


def reference(x, W, A, B, ids, scales, bias, act, residual):
    M, K = x.shape
    rank = A.shape[1]
    x64 = x.to(F64)
    v = x64 @ W.to(F64).t()
    step = (K / 16 + 48) * 2.0 ** -23
    e = step * (x64.abs() @ W.to(F64).abs().t())
    for m, a in enumerate(ids.tolist()):
        if 0 <= a < A.shape[0]:
            c = 1.0 if scales is None else scales[a].to(F64)
            A64, B64 = A[a].to(F64), B[a].to(F64)
            t = c * (A64 @ x64[m])
            d = B64 @ t
            e[m] += c * step * (B64.abs() @ (A64.abs() @ x64[m].abs()))
            e[m] += 2.0 ** -23 * ((rank + 4) * (B64.abs() @ t.abs()) + v[m].abs() + d.abs())
            v[m] += d
    if bias is not None:
        v = v + bias.to(F64)
    want = activate(v, act)
    tol = 1.13 * e + 2.0 ** -20 * v.abs()
    if residual is not None:
        want = want + residual.to(F64)
        tol = tol + 2.0 ** -23 * want.abs()
    return want, tol + HALF_BF16 * (want.abs() + tol)


# Whole and split tiles, every padded row count, ragged N and K, the 64-row finish, more
# tiles than CTAs; every rank class (one half step, whole steps, the largest).
SHAPES = [(1, 16, 64, 8), (1, 1, 8, 16), (3, 200, 136, 24), (5, 4099, 1000, 8), (16, 640, 7168, 16),
          (17, 256, 4096, 64), (32, 1001, 1024, 128), (33, 300, 1000, 40), (64, 1024, 7168, 16), (64, 129, 72, 128),
          (20, 18432, 512, 32), (40, 20480, 512, 16), (64, 20480, 256, 64), (63, 7161, 520, 16)]


@pytest.mark.parametrize("M,N,K,rank", SHAPES)
@pytest.mark.parametrize("kind", ["own", "pairs", "some"])
@pytest.mark.parametrize("pdl", [False, True])
def test_integer_inputs_bit_exact(cuda_ok, M, N, K, rank, kind, pdl):
    E = min(M, 11)
    x, W = gemm_inputs_device(M, N, K, workloads.seed_for("lora", M, N, K), kind="int")
    A, B, scales = pool(E, rank, N, K, M + N, "int")
    ids = adapter_ids(M, E, kind, 3)
    bias, res = extras(M, N, 5, "int")
    got = run(x, W, A, B, ids, scales, bias, "relu", res, in_place=pdl, pdl=pdl)
    want, _ = reference(x, W, A, B, ids, scales, bias, "relu", res)
    assert want.abs().max() < 2 ** 24
    assert torch.equal(got, want.float().to(BF))


@pytest.mark.parametrize("M,N,K,rank", [(1, 2048, 7168, 16), (5, 4099, 1000, 8), (16, 18432, 7168, 64),
                                        (64, 7168, 18432, 16), (33, 300, 1000, 24), (64, 20480, 1024, 128)])
@pytest.mark.parametrize("kind", ["own", "one", "last"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
def test_against_64_bits(cuda_ok, M, N, K, rank, kind, act):
    E = min(M, 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF)
    W = (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).to(BF)
    A, B, scales = pool(E, rank, N, K, M + K)
    ids = adapter_ids(M, E, kind, 4)
    bias, res = extras(M, N, 6)
    if act == "none":
        scales, bias = None, None
    got = run(x, W, A, B, ids, scales, bias, act, res)
    want, tol = reference(x, W, A, B, ids, scales, bias, act, res)
    check_close(got, want, tol, f"{kind} {act}")
    again = run(x, W, A, B, ids, scales, bias, act, res, pdl=True)
    assert torch.equal(again.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("M,N,K", [(4, 300, 512), (16, 18432, 256), (64, 1024, 4096), (40, 20480, 512)])
def test_rows_without_an_adapter_have_the_epilogue_bits(cuda_ok, M, N, K):
    x, W = gemm_inputs_device(M, N, K, workloads.seed_for("lora0", M, N, K))
    A, B, scales = pool(3, 16, N, K, 9)
    bias, res = extras(M, N, 7)
    want = torch.empty(M, N, dtype=BF, device="cuda")
    sk.decode_gemm_bf16_epilogue(x, W, want, bias, "gelu", res)
    for kind in ("none", "some"):
        ids = adapter_ids(M, 3, kind, 1)
        got = run(x, W, A, B, ids, scales, bias, "gelu", res)
        bare = ids < 0
        assert torch.equal(got[bare].view(torch.int16), want[bare].view(torch.int16))


def test_unused_adapters_are_not_read(cuda_ok):
    """NaN in the adapters that no row has, and a finite result; one out of range is none."""
    M, N, K, rank = 9, 640, 1000, 16
    x, W = gemm_inputs_device(M, N, K, 21)
    A, B, scales = pool(5, rank, N, K, 22)
    for a in (0, 2, 4):
        A[a], B[a], scales[a] = float("nan"), float("nan"), float("nan")
    ids = torch.tensor([1, 3, -1, 1, 3, 3, -2147483648, 1, -1], dtype=torch.int32, device="cuda")
    got = run(x, W, A, B, ids, scales)
    want, tol = reference(x, W, A, B, ids, scales, None, "none", None)
    check_close(got, want, tol, "unused")
    bad = ids.clone()
    bad[4], bad[0] = 5, 2147483647
    out = torch.empty_like(got)
    sk.decode_gemm_bf16_lora(x, W, out, A, B, bad, scales)
    st, word = sk.device_error()
    assert sk.STATUS[st] == "SKINNY_ERR_INDEX" and word == 256
    bad[4], bad[0] = -1, -1
    assert torch.equal(out, run(x, W, A, B, bad, scales))


def test_linears_one_after_another_replayed(cuda_ok):
    """Up and down with adapters, each reading what the kernel before wrote, with and without
    programmatic dependent launch, and as a graph whose inputs and adapters change."""
    M, H, F, rank, E = 12, 1024, 4096, 16, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(M, H, generator=g, device="cuda").to(BF)
    W1 = (torch.randn(F, H, generator=g, device="cuda") * H ** -0.5).to(BF)
    W2 = (torch.randn(H, F, generator=g, device="cuda") * F ** -0.5).to(BF)
    A1, B1, s1 = pool(E, rank, F, H, 3)
    A2, B2, s2 = pool(E, rank, H, F, 4)
    ids = adapter_ids(M, E, "some", 5)
    h, y = torch.empty(M, F, dtype=BF, device="cuda"), torch.empty(M, H, dtype=BF, device="cuda")

    def step(pdl):
        sk.decode_gemm_bf16_lora(x, W1, h, A1, B1, ids, s1, activation="silu", pdl=pdl)
        sk.decode_gemm_bf16_lora(h, W2, y, A2, B2, ids, s2, residual=x, pdl=pdl)
        for _ in range(4):  # what one call leaves in the scratch is another's when it runs
            sk.decode_gemm_bf16_lora(y, W1, h, A1, B1, ids, s1, activation="relu", pdl=pdl)
            sk.decode_gemm_bf16_lora(h, W2, y, A2, B2, ids, s2, residual=y, pdl=pdl)
    step(False)
    first = y.clone()
    for _ in range(3):
        step(True)
        assert torch.equal(y, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(True)
    graph.replay()
    assert torch.equal(y, first)
    x.copy_(torch.randn(M, H, generator=g, device="cuda").to(BF))
    ids.copy_(adapter_ids(M, E, "own", 6))
    graph.replay()
    second = y.clone()
    step(False)
    assert torch.equal(y, second) and not torch.equal(y, first)


def test_a_pool_past_32_bits(cuda_ok):
    """Adapters whose elements lie past 2^31."""
    N, K, rank = 20480, 64, 128
    E = (1 << 31) // (N * rank) + 3
    B = torch.zeros(E, N, rank, dtype=BF, device="cuda")
    A = torch.zeros(E, rank, K, dtype=BF, device="cuda")
    B[E - 1], A[E - 1] = 1.0, 0.5
    B[E - 2, :, 0], A[E - 2, 0] = 2.0, 1.0
    x = torch.ones(3, K, dtype=BF, device="cuda")
    W = torch.zeros(N, K, dtype=BF, device="cuda")
    ids = torch.tensor([E - 1, 0, E - 2], dtype=torch.int32, device="cuda")
    got = run(x, W, A, B, ids)
    assert (got[0] == 128 * 32).all() and (got[1] == 0).all() and (got[2] == 128).all()
