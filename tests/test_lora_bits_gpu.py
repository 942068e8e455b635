"""decode_gemm_bf16_lora on the GPU: the same rows, weight and adapters give the same bits with and
without programmatic dependent launch and whatever other adapters the pool holds, by whichever of
its two forms the call goes."""
import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
from test_lora_gpu import BF, adapter_ids, pool, run

pytestmark = pytest.mark.gpu


def inputs(M, N, K, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF)
    return x, (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).to(BF)


# Less than 1 MiB of weight a CTA for up to 32 rows (the shallow ring with dependent launch, the deep
# one without), and more; whole tiles and split ones; ranks of either form and on the border.
@pytest.mark.parametrize("M,N,K,rank", [(32, 1001, 1024, 128), (24, 2048, 4096, 64), (17, 300, 2056, 72), (20, 640, 512, 32),
                                        (32, 20480, 512, 96), (30, 4099, 7168, 24), (16, 2048, 4096, 128), (64, 2048, 4096, 48)])
@pytest.mark.parametrize("kind,E", [("own", 64), ("pairs", 4), ("one", 2), ("some", 9)])
def test_dependent_launch_and_the_pool_leave_the_bits(cuda_ok, M, N, K, rank, kind, E):
    x, W = inputs(M, N, K, M + K)
    A, B, scales = pool(E, rank, N, K, M + N)
    ids = adapter_ids(M, E, kind, 5)
    want = run(x, W, A, B, ids, scales)
    for pdl in (True, False):
        assert torch.equal(run(x, W, A, B, ids, scales, pdl=pdl).view(torch.int16), want.view(torch.int16)), pdl
    more = 300 - E  # the same adapters at the end of a larger pool
    big = [torch.cat([torch.ones(more, *t.shape[1:], dtype=t.dtype, device="cuda"), t]) for t in (A, B, scales)]
    for pdl in (True, False):
        got = run(x, W, big[0], big[1], torch.where(ids >= 0, ids + more, ids), big[2], pdl=pdl)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), pdl
