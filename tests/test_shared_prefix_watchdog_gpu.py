"""The bounded waits of decode_attention_shared_prefix_bf16 on the GPU: a wait that can never
complete ends with a recorded status, nothing of the call is left behind (copies in flight,
tensor memory, counters in the workspace), and the next call with the same workspace has the
same bits as the one before. Nothing here faults or traps."""
import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
from test_shared_prefix_gpu import Case

pytestmark = pytest.mark.gpu

WAIT_BIT = 512


def selftest(c, ws, timeout_ns):
    sk.shared_prefix_selftest(c.q, c.k, c.v, c.prefix_table, c.prefix_length, c.table, c.lengths, c.out, c.lse, ws,
                              timeout_ns)


# One and two tiles of query rows; rings of an even (64, 128) and an odd number of stages (192: 7,
# 256: 5); boxes, and pages that are copied token by token.
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("R,page", [(3, 16), (40, 16), (40, 12)])
def test_a_wait_that_runs_out_is_reported_and_leaves_nothing_behind(cuda_ok, D, R, page):
    c = Case(R, 8, 1, D, page, 5000, 40, seed=D + R)
    ws = sk.shared_prefix_workspace(R, 8, 1, D)
    c.check(workspace=ws)
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(2):
        selftest(c, ws, 2_000_000)  # 2 ms
        torch.cuda.synchronize()
        status, word = sk.device_error()
        assert status == 9, sk.status_string(status)
        assert word == WAIT_BIT
        assert sk.device_error() == (0, 0)
        c.call(workspace=ws)
        assert sk.device_error() == (0, 0)
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


def test_limits_out_of_range_are_refused(cuda_ok):
    c = Case(3, 8, 1, 64, 16, 100, 4)
    ws = sk.shared_prefix_workspace(3, 8, 1, 64)
    for bad in (0, 999, 3_000_000_000):
        with pytest.raises(sk.SkinnyError) as e:
            selftest(c, ws, bad)
        assert sk.STATUS[e.value.status] == "SKINNY_ERR_ARG"
    assert sk.device_error() == (0, 0)
