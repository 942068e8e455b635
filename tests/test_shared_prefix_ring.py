"""The ring of the attention over a shared prefix and the refusals of its self-test, without a GPU."""
import os
import subprocess

import skinny_bf16_gemm_gb300 as sk
from test_attention_abi import ALIAS, ALIGN, ARG, DEVICE, MB, NULL, SHAPE, cache_at, lib, mem  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))


def test_no_unit_of_the_ring_meets_another(tmp_path):
    """tests/native/prefix_ring_check.cpp with the host compiler. It also runs a ring whose stages
    keys and values take in turn and one that waits for half its units at the end, and must find
    that for an odd number of stages the one is unsafe and the other misses copies."""
    program = str(tmp_path / "ring")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(sk.PKG, "csrc"), "-x", "c++",
                    os.path.join(HERE, "native", "prefix_ring_check.cpp"), "-o", program], check=True, timeout=300)
    p = subprocess.run([program], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout == "ok\n", p.stdout


def test_the_selftest_checks_its_limit_and_arguments_before_cuda(lib, mem):  # noqa: F811
    _, p = mem
    size = lib.skinny_shared_prefix_workspace_bytes(3, 4, 2, 64, 152)
    ok = dict(q=p, q_stride=256, rows=3, q_heads=4, prefix_table=p + MB, prefix_width=6, prefix_length=p + MB + 4096,
              block_table=p + 2 * MB, table_stride=4, table_width=4, lengths=p + 3 * MB, scale=0.125, out=p + 4 * MB,
              lse=p + 5 * MB, workspace=p + 8 * MB, workspace_bytes=size)

    def call(timeout_ns=10 ** 6, **kw):
        a = sk.SharedPrefixAttentionArgs(**dict(ok, **kw))
        a.cache = cache_at(p + 6 * MB, v=p + 7 * MB)
        return lib.skinny_shared_prefix_selftest(bytes(a), timeout_ns, None)
    for bad in (0, 999, 3_000_000_000, -1):
        assert call(bad) == ARG
    assert call(q=None) == NULL and call(rows=0) == SHAPE and call(q=p + 8) == ALIGN and call(out=p) == ALIAS
    assert lib.skinny_shared_prefix_selftest(None, 10 ** 6, None) == NULL
    import torch
    if not torch.cuda.is_available():
        assert call() == DEVICE
