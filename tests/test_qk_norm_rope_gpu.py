"""qk_norm_rope_bf16 on the GPU against the definition in 64 bits (tolerances:
attention_helpers.norm_rope_reference); values and cache rows bit for bit."""
import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
from attention_helpers import check_close, make_cache, norm_rope_reference, rope_table
from gpu_helpers import Guarded

pytestmark = pytest.mark.gpu
MAX_POS = 5000


def inputs(M, Hq, Hkv, D, rot, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    qkv = (randn(M, (Hq + 2 * Hkv) * D) * 2).to(torch.bfloat16)
    qg, kg = (1 + 0.2 * randn(D)).to(torch.bfloat16), (1 + 0.2 * randn(D)).to(torch.bfloat16)
    pos = torch.randint(0, MAX_POS, (M,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = MAX_POS - 1
    return qkv, qg, kg, rope_table(MAX_POS, rot) if rot else None, pos


def run_and_check(M, Hq, Hkv, D, rot, interleaved=False, page=16, layout="nhd", norm=(True, True), seed=0):
    qkv, qg, kg, rope, pos = inputs(M, Hq, Hkv, D, rot, seed)
    qg, kg = qg if norm[0] else None, kg if norm[1] else None
    pages = M // page + 3
    k, v = make_cache(pages, page, Hkv, D, layout, seed + 1)
    k0, v0 = k.clone(), v.clone()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 2)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:M]
    slots[M // 2] = -1
    q_out, k_out = Guarded((M, Hq, D)), Guarded((M, Hkv, D))
    sk.qk_norm_rope_bf16(qkv, Hq, Hkv, qg, kg, rope, pos, q_out.tensor, k_out.tensor, k, v, slots,
                         interleaved=interleaved)
    torch.cuda.synchronize()
    q_out.check(), k_out.check()
    assert sk.device_error() == (0, 0)
    x = qkv.view(M, Hq + 2 * Hkv, D)
    for got, heads, gamma, name in ((q_out.tensor, x[:, :Hq], qg, "q"),
                                    (k_out.tensor, x[:, Hq:Hq + Hkv], kg, "k")):
        want, tol = norm_rope_reference(heads, gamma, rope, pos, interleaved, 1e-6)
        check_close(got, want, tol, name)
    # The cache: each row's key as in k_out, its value unchanged, nothing else touched.
    for r, s in enumerate(slots.tolist()):
        if s >= 0:
            k0[s // page, s % page], v0[s // page, s % page] = k_out.tensor[r], x[r, Hq + Hkv:]
    assert torch.equal(k, k0) and torch.equal(v, v0)


@pytest.mark.parametrize("D,rot", [(8, 0), (16, 16), (64, 64), (64, 32), (72, 48), (80, 80), (96, 96), (112, 16),
                                   (128, 128), (128, 64), (192, 64), (256, 256), (256, 128), (248, 240)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_widths(cuda_ok, D, rot, interleaved):
    run_and_check(19, 6, 2, D, rot, interleaved, seed=D + rot)


@pytest.mark.parametrize("M,Hq,Hkv", [(1, 1, 1), (1, 7, 1), (1, 56, 8), (2, 5, 3), (64, 56, 8), (333, 7, 1),
                                      (1500, 32, 8), (70, 200, 40)])
def test_rows_and_heads(cuda_ok, M, Hq, Hkv):
    """From one row to enough for four heads a lane group (and heads past one block)."""
    run_and_check(M, Hq, Hkv, 128, 128, seed=M)


@pytest.mark.parametrize("page,layout", [(1, "nhd"), (7, "hnd"), (64, "kv"), (16, "padded"), (24, "hnd")])
def test_layouts(cuda_ok, page, layout):
    run_and_check(50, 4, 2, 64, 64, page=page, layout=layout)


@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("rot", [0, 64])
def test_without_norm_or_rotation(cuda_ok, norm, rot):
    run_and_check(21, 6, 2, 64, rot, norm=norm)


def test_in_place_equals_out_of_place(cuda_ok):
    M, Hq, Hkv, D = 40, 7, 2, 96
    qkv, qg, kg, rope, pos = inputs(M, Hq, Hkv, D, D)
    q, k = torch.empty(M, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(
        M, Hkv, D, dtype=torch.bfloat16, device="cuda")
    sk.qk_norm_rope_bf16(qkv, Hq, Hkv, qg, kg, rope, pos, q, k)
    wide = torch.full((M, qkv.shape[1] + 40), 3.0, dtype=torch.bfloat16, device="cuda")
    rows = wide[:, 8:8 + qkv.shape[1]]
    rows.copy_(qkv)
    qv = rows[:, :Hq * D].view(M, Hq, D)
    kv = rows[:, Hq * D:(Hq + Hkv) * D].view(M, Hkv, D)
    sk.qk_norm_rope_bf16(rows, Hq, Hkv, qg, kg, rope, pos, qv, kv)
    torch.cuda.synchronize()
    assert torch.equal(qv, q) and torch.equal(kv, k)
    assert torch.equal(rows[:, (Hq + Hkv) * D:], qkv[:, (Hq + Hkv) * D:])
    assert (wide[:, :8] == 3).all() and (wide[:, 8 + qkv.shape[1]:] == 3).all()


def test_far_positions_and_zero_rows(cuda_ok):
    """A zero head stays zero (eps keeps the root finite); a huge one is normalised."""
    M, Hq, Hkv, D = 4, 2, 1, 64
    qkv, qg, kg, rope, pos = inputs(M, Hq, Hkv, D, D)
    qkv[0] = 0
    qkv[1] *= 2.0 ** 60
    q = torch.empty(M, Hq, D, dtype=torch.bfloat16, device="cuda")
    sk.qk_norm_rope_bf16(qkv, Hq, Hkv, qg, kg, rope, pos, q)
    torch.cuda.synchronize()
    assert not q[0].any()
    want, tol = norm_rope_reference(qkv.view(M, -1, D)[1:, :Hq], qg, rope, pos[1:], False, 1e-6)
    check_close(q[1:], want, tol, "q")


def test_bad_positions_and_slots_are_reported_and_not_written(cuda_ok):
    M, Hq, Hkv, D, page = 6, 3, 1, 64, 8
    qkv, qg, kg, rope, pos = inputs(M, Hq, Hkv, D, D)
    k, v = make_cache(4, page, Hkv, D, "nhd", 3)
    k0, v0 = k.clone(), v.clone()
    pos[1], pos[2] = MAX_POS, -1
    slots = torch.tensor([0, 1, 2, 32, -9, 2 ** 40], device="cuda")
    q = torch.full((M, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    sk.qk_norm_rope_bf16(qkv, Hq, Hkv, qg, kg, rope, pos, q, k_cache=k, v_cache=v, slots=slots)
    assert sk.device_error() == (11, 256)
    assert sk.device_error() == (0, 0)
    want, tol = norm_rope_reference(qkv.view(M, -1, D)[:, :Hq], qg, rope, pos.clamp(0, MAX_POS - 1), False, 1e-6)
    for r in (0, 4):
        check_close(q[r], want[r], tol[r], "q")
    for r in (1, 2, 3, 5):
        assert (q[r] == 5).all()
    assert not torch.equal(k[0, 0], k0[0, 0]) and torch.equal(v[0, 0], qkv.view(M, -1, D)[0, Hq + Hkv:])
    k[0, 0], v[0, 0] = k0[0, 0], v0[0, 0]
    assert torch.equal(k, k0) and torch.equal(v, v0)


def test_bad_rows_among_many(cuda_ok):
    """Blocks that go through many rows leave the bad ones out and go on."""
    M, Hq, Hkv, D, page = 5000, 7, 1, 128, 16
    qkv, qg, kg, rope, pos = inputs(M, Hq, Hkv, D, D)
    k, v = make_cache(M // page + 1, page, Hkv, D, "nhd", 3)
    k0 = k.clone()
    slots = torch.arange(M, device="cuda")
    bad = torch.arange(3, M, 7, device="cuda")
    pos[bad[::2]] = -5
    slots[bad[1::2]] = 2 ** 33
    q = torch.full((M, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    sk.qk_norm_rope_bf16(qkv, Hq, Hkv, qg, kg, rope, pos, q, k_cache=k, v_cache=v, slots=slots)
    assert sk.device_error() == (11, 256)
    good = torch.ones(M, dtype=torch.bool, device="cuda")
    good[bad] = False
    x = qkv.view(M, -1, D)
    want, tol = norm_rope_reference(x[:, :Hq], qg, rope, pos.clamp(0), False, 1e-6)
    check_close(q[good], want[good], tol[good], "q")
    assert (q[bad] == 5).all()
    want, tol = norm_rope_reference(x[:, Hq:Hq + Hkv], kg, rope, pos.clamp(0), False, 1e-6)
    flat, flat0 = k.view(-1, Hkv, D)[:M], k0.view(-1, Hkv, D)[:M]
    check_close(flat[good], want[good], tol[good], "k")
    assert torch.equal(flat[bad], flat0[bad])


def test_slots_past_32_bits(cuda_ok):
    """The last page starts 8 GB into the pool."""
    D, page, step = 64, 16, (1 << 31) + 64
    pool = torch.zeros(2 * step + 4 * page * D, dtype=torch.bfloat16, device="cuda")
    k = pool.as_strided((3, page, 1, D), (step, D, D, 1))
    v = torch.empty(3, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(2 * step + 4 * page * D, dtype=torch.bfloat16, device="cuda").as_strided(
        (3, page, 1, D), (step, D, D, 1))
    qkv, qg, kg, rope, pos = inputs(2, 2, 1, D, D)
    q, ko = torch.empty(2, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(
        2, 1, D, dtype=torch.bfloat16, device="cuda")
    sk.qk_norm_rope_bf16(qkv, 2, 1, qg, kg, rope, pos, q, ko, k, v, torch.tensor([47, 3], device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(k[2, 15], ko[0]) and torch.equal(k[0, 3], ko[1])
    assert torch.equal(v[2, 15, 0], qkv[0, -D:]) and torch.equal(v[0, 3, 0], qkv[1, -D:])
    assert int((pool != 0).sum()) == int((ko != 0).sum())


def test_captured_and_replayed_with_pdl(cuda_ok):
    M, Hq, Hkv, D = 9, 7, 1, 128
    qkv, qg, kg, rope, pos = inputs(M, Hq, Hkv, D, D)
    q, want = (torch.empty(M, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sk.qk_norm_rope_bf16(qkv, Hq, Hkv, qg, kg, rope, pos, q, pdl=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sk.qk_norm_rope_bf16(qkv, Hq, Hkv, qg, kg, rope, pos, q, pdl=True)
    qkv.copy_(qkv.flip(0))
    pos.copy_(pos.flip(0))
    g.replay()
    sk.qk_norm_rope_bf16(qkv, Hq, Hkv, qg, kg, rope, pos, want)
    torch.cuda.synchronize()
    assert torch.equal(q, want)
