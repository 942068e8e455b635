"""The ring of the attention over a shared prefix, checked by itself without a GPU."""
import os
import subprocess

import skinny_bf16_gemm_gb300 as sk

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
