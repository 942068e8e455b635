"""decode_gemm_bf16_epilogue on the GPU.

Integer inputs without a curved activation are exact in FP32 whatever the summation order
and must match bit for bit. Otherwise, against 64 bits: the FP32 sum over K is taken in
steps of 16 products, each step off by at most 2^-23 (truncation allowed for) of the
running magnitude, so e = (K / 16 + 16) 2^-23 sum |x w|; the activations' slopes are at
most 1.13 and their own roundings a few FP32 steps of |v|; then half a BF16 step."""
import math

import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
import workloads
from attention_helpers import F64, HALF_BF16, check_close
from gpu_helpers import Guarded, gemm_inputs_device

pytestmark = pytest.mark.gpu


def activate(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def extras(M, N, seed, kind="normal"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if kind == "int":
        return (torch.randint(-9, 10, (N,), generator=g, device="cuda").to(torch.bfloat16),
                torch.randint(-99, 100, (M, N), generator=g, device="cuda").to(torch.bfloat16))
    return (torch.randn(N, generator=g, device="cuda").to(torch.bfloat16),
            torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16))


def run(x, W, bias, act, residual, in_place=False, **kw):
    M, N = x.shape[0], W.shape[0]
    out = Guarded((M, N), fill=residual if in_place else None)
    sk.decode_gemm_bf16_epilogue(x, W, out.tensor, bias, act, out.tensor if in_place else residual, **kw)
    torch.cuda.synchronize()
    out.check()
    assert sk.device_error() == (0, 0)
    return out.tensor


# Split and whole tiles, every padded row count, ragged N and K, the 64-row finish kernel
# (64 x 1024 and 48 x 300), more tiles than CTAs (N = 20480), staged whole tiles (N = 18432).
SHAPES = [(1, 16, 64), (1, 1, 8), (3, 200, 136), (5, 4099, 1000), (16, 640, 7168), (17, 256, 4096),
          (32, 1001, 1024), (33, 300, 1000), (48, 300, 2048), (64, 1024, 7168), (64, 129, 72), (20, 18432, 512),
          (64, 18432, 256), (40, 20480, 512), (64, 7168, 1000), (63, 7161, 520)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("in_place", [False, True])
def test_integer_inputs_bit_exact(cuda_ok, M, N, K, act, in_place):
    x, W = gemm_inputs_device(M, N, K, workloads.seed_for("epi", M, N, K), kind="int")
    bias, res = extras(M, N, 5, "int")
    got = run(x, W, bias, act, res, in_place)
    want = activate(x.to(F64) @ W.to(F64).t() + bias.to(F64), act) + res.to(F64)
    assert want.abs().max() < 2 ** 24
    assert torch.equal(got, want.float().to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(1, 2048, 7168), (5, 4099, 1000), (16, 18432, 7168), (64, 7168, 18432),
                                   (33, 300, 1000), (64, 20480, 1024)])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("with_bias,with_res", [(True, False), (False, True), (True, True)])
def test_against_64_bits(cuda_ok, M, N, K, act, with_bias, with_res):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(N, K, generator=g, device="cuda") * (1.5 * K ** -0.5)).to(torch.bfloat16)
    bias, res = extras(M, N, 6)
    got = run(x, W, bias if with_bias else None, act, res if with_res else None, pdl=(M == 16) or None)
    v = x.to(F64) @ W.to(F64).t()
    e = (K / 16 + 16) * 2.0 ** -23 * (x.abs().to(F64) @ W.abs().to(F64).t())
    if with_bias:
        v = v + bias.to(F64)
    want = activate(v, act)
    tol = 1.13 * e + 2.0 ** -20 * v.abs()
    if with_res:
        want = want + res.to(F64)
        tol = tol + 2.0 ** -23 * want.abs()
    check_close(got, want, tol + HALF_BF16 * (want.abs() + tol), act)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_plain_call_has_the_gemm_bits(cuda_ok, M, N, K):
    x, W = gemm_inputs_device(M, N, K, workloads.seed_for("epi0", M, N, K))
    want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    sk.decode_gemm_bf16(x, W, want)
    assert torch.equal(run(x, W, None, "none", None).view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("M,N,K", [(8, 65536, 64), (64, 50001, 128), (31, 40000, 200), (64, 40000, 1000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_many_tiles_a_cta(cuda_ok, M, N, K, in_place):
    """Several tiles a CTA: whole ones between the split ends, both accumulators in turn."""
    x, W = gemm_inputs_device(M, N, K, workloads.seed_for("epi2", M, N, K), kind="int")
    bias, res = extras(M, N, 8, "int")
    got = run(x, W, bias, "relu", res, in_place)
    want = activate(x.to(F64) @ W.to(F64).t() + bias.to(F64), "relu") + res.to(F64)
    assert torch.equal(got, want.float().to(torch.bfloat16))


def test_activation_tails(cuda_ok):
    """Sums from -200 to 200 through each activation: no NaN where exp or its inverse
    overflows."""
    N, K = 401, 8
    x = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    bias = torch.linspace(-200, 200, N, device="cuda").to(torch.bfloat16)
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        got = run(x, W, bias, act, None)
        v = bias.to(F64)[None]
        want = activate(v, act)
        # Below about -88 silu's exp overflows to inf and gives -0 for a value under 1e-36.
        tol = HALF_BF16 * want.abs() + 2.0 ** -20 * v.abs()
        check_close(got, want, tol, act)


def test_chained_on_one_stream_with_pdl(cuda_ok):
    """Up with an activation, down with the residual in place, replayed as a graph."""
    M, H, F = 16, 1024, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16)
    W1 = (torch.randn(F, H, generator=g, device="cuda") * H ** -0.5).to(torch.bfloat16)
    W2 = (torch.randn(H, F, generator=g, device="cuda") * F ** -0.5).to(torch.bfloat16)
    b = torch.randn(F, generator=g, device="cuda").to(torch.bfloat16)
    h, y, y0 = (torch.empty(M, n, dtype=torch.bfloat16, device="cuda") for n in (F, H, H))
    sk.decode_gemm_bf16_epilogue(x, W1, h, b, "silu")
    sk.decode_gemm_bf16_epilogue(h, W2, y0, residual=x)

    def step(pdl):
        y.copy_(x)
        for _ in range(1):
            sk.decode_gemm_bf16_epilogue(x, W1, h, b, "silu", pdl=pdl)
            sk.decode_gemm_bf16_epilogue(h, W2, y, residual=y, pdl=pdl)
    for pdl in (False, True):
        step(pdl)
        assert torch.equal(y, y0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(True)
    y.zero_()
    graph.replay()
    assert torch.equal(y, y0)
