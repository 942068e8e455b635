"""decode_attention_bf16 on the GPU against the definition in 64 bits. The tolerances are
derived in attention_helpers.attention_reference."""
import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
from attention_helpers import attention_reference, check_close, make_cache
from gpu_helpers import Guarded

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def setup(lengths, Hq, Hkv, D, page, layout="nhd", seed=0, width=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    width = width or max(1, -(-max(max(lengths), 1) // page))
    R = len(lengths)
    pages = R * width + 3
    k, v = make_cache(pages, page, Hkv, D, layout, seed)
    table = torch.randperm(pages, generator=g, device="cuda")[:R * width].view(R, width).to(torch.int32)
    q = (torch.randn(R, Hq, D, generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    return q, k, v, table, ints(lengths)


def run_and_check(q, k, v, table, lengths, window=0, sinks=0, scale=None, workspace=None):
    R, Hq, D = q.shape
    out = Guarded((R, Hq, D))
    lse = torch.full((R, Hq), 7.0, dtype=torch.float32, device="cuda")
    sk.decode_attention_bf16(q, k, v, table, lengths, out.tensor, scale=scale, window=window, sinks=sinks,
                             lse=lse, workspace=workspace)
    torch.cuda.synchronize()
    out.check()
    assert sk.device_error() == (0, 0)
    want, want_lse, tol, lse_tol = attention_reference(q, k, v, table, lengths,
                                                       D ** -0.5 if scale is None else scale, window, sinks)
    check_close(out.tensor, want, tol, "out")
    check_close(lse, want_lse, lse_tol, "lse")
    return out.tensor, lse


RAGGED = [130, 0, 1, 15, 16, 17, 63, 64, 65, 200, 1000, 333]


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (8, 8), (24, 2), (40, 1), (33, 1), (64, 4)])
def test_heads_and_widths(cuda_ok, D, Hq, Hkv):
    """Every head width with groups of 1 to 40 heads: one, two and four blocks of 8, and
    groups cut into several blocks; ragged rows, one of them empty."""
    run_and_check(*setup(RAGGED, Hq, Hkv, D, 16, seed=D + Hq))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 256])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv", "padded"])
def test_pages_and_layouts(cuda_ok, page, layout):
    run_and_check(*setup(RAGGED, 14, 2, 128, page, layout, seed=page))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 4), (63, 0), (128, 100), (1000, 1),
                                          (5000, 10), (17, 1000)])
def test_window_and_sinks(cuda_ok, window, sinks):
    run_and_check(*setup(RAGGED, 8, 2, 64, 16, seed=window), window=window, sinks=sinks)


@pytest.mark.parametrize("R,n,Hq,Hkv,D", [(1, 1, 7, 1, 128), (1, 64, 7, 1, 128), (1, 65, 1, 1, 64),
                                          (1, 20000, 7, 1, 128), (1, 20000, 32, 8, 64), (2, 9999, 16, 1, 256),
                                          (3, 5000, 32, 1, 128), (1, 131071, 8, 1, 64), (5, 2000, 3, 3, 96)])
def test_long_rows_are_split_and_joined(cuda_ok, R, n, Hq, Hkv, D):
    """From one tile to many CTAs a head: one and two levels of joins."""
    run_and_check(*setup([n] * R, Hq, Hkv, D, 64, seed=n))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (14, 2, 128), (16, 1, 256), (32, 1, 128), (8, 1, 192), (4, 1, 64)])
@pytest.mark.parametrize("parts", [19, 20, 21, 26, 37])
def test_joins_around_the_second_level(cuda_ok, parts, Hq, Hkv, D):
    """A row of about so many chunks a key head, 8 tiles each; two key heads meet in a chunk."""
    tile = 32 if Hq // Hkv <= 8 and D <= 128 else 16
    run_and_check(*setup([parts * 8 * tile - 3], Hq, Hkv, D, 64, seed=parts))


def test_many_rows(cuda_ok):
    """1024 rows, from empty to a few tiles; the fused table is wider than any row."""
    g = torch.Generator()
    g.manual_seed(5)
    lengths = torch.randint(0, 150, (1024,), generator=g).tolist()
    lengths[0] = lengths[500] = lengths[1023] = 0
    run_and_check(*setup(lengths, 4, 2, 64, 32, seed=9, width=9))


@pytest.mark.parametrize("lengths", [[0], [0, 0, 0], [0, 5, 0], [1, 1, 1]])
def test_empty_rows(cuda_ok, lengths):
    out, lse = run_and_check(*setup(lengths, 6, 2, 128, 16))
    for r, n in enumerate(lengths):
        if n == 0:
            assert not out[r].any() and torch.isinf(lse[r]).all()


def test_one_token_returns_its_value_exactly(cuda_ok):
    q, k, v, table, lengths = setup([1, 1, 1], 4, 2, 64, 8)
    out, _ = run_and_check(q, k, v, table, lengths)
    want = v[table[:, 0].long(), 0].repeat_interleave(2, dim=1)
    assert torch.equal(out, want)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(cuda_ok, scale):
    run_and_check(*setup([50, 300, 7], 5, 1, 64, 16), scale=scale)


def test_queries_strided_in_place_of_the_qkv_rows(cuda_ok):
    q, k, v, table, lengths = setup([40, 300, 5], 6, 2, 64, 16)
    wide = torch.full((3, 10 * 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = wide[:, :6 * 64].view(3, 6, 64)
    view.copy_(q)
    a, _ = run_and_check(view, k, v, table, lengths)
    b, _ = run_and_check(q, k, v, table, lengths)
    assert torch.equal(a, b)


def test_unseen_pages_and_tokens_are_not_read(cuda_ok):
    """Pages between the sinks and the window have no valid table entry, and everything a
    row does not see is NaN."""
    page, n, window, sinks = 16, 400, 70, 5
    q, k, v, table, lengths = setup([n, 3], 4, 2, 64, page)
    poison_k, poison_v = torch.full_like(k, float("nan")), torch.full_like(v, float("inf"))
    for r, m in enumerate([n, 3]):
        for j in range(m):
            if j < sinks or j >= m - window:
                at, off = int(table[r, j // page]), j % page
                poison_k[at, off], poison_v[at, off] = k[at, off], v[at, off]
    clean = table.clone()
    want, _ = run_and_check(q, k, v, clean, lengths, window=window, sinks=sinks)
    table[0, 1:(n - window) // page] = -1
    table[1, 1:] = 2 ** 30
    out = torch.empty_like(q)
    sk.decode_attention_bf16(q, poison_k, poison_v, table, lengths, out, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert sk.device_error() == (0, 0)
    assert torch.equal(out, want)


def test_bad_pages_and_lengths_are_reported_and_left_out(cuda_ok):
    """A page out of range counts as not seen, a length past the table as the table's end,
    a negative one as zero; the device word says so once."""
    page = 16
    q, k, v, table, lengths = setup([64, 40, 30], 4, 2, 64, page)
    good_out = torch.empty_like(q)
    sk.decode_attention_bf16(q, k, v, table, lengths, good_out)
    assert sk.device_error() == (0, 0)
    bad = table.clone()
    bad[0, 1] = -1
    bad[0, 3] = k.shape[0]
    out = torch.empty_like(q)
    sk.decode_attention_bf16(q, k, v, bad, lengths, out)
    st, word = sk.device_error()
    assert st == 11 and word == 256
    assert sk.device_error() == (0, 0)
    # Row 0 sees pages 0 and 2 only; the others are as before.
    short = table.clone()
    short[0, 1] = table[0, 2]
    n = ints([32, 40, 30])
    want, _, tol, _ = attention_reference(q, k, v, short, n, 64 ** -0.5)
    check_close(out, want, tol, "out")
    assert torch.equal(out[1:], good_out[1:])
    sk.decode_attention_bf16(q, k, v, table, ints([70, -5, 30]), out)
    assert sk.device_error() == (11, 256)
    assert torch.equal(out[0], good_out[0]) and not out[1].any() and torch.equal(out[2], good_out[2])
    table.fill_(-7)
    sk.decode_attention_bf16(q, k, v, table, lengths, out)
    assert sk.device_error() == (11, 256)
    assert not out.any()


def test_nan_and_infinite_scores(cuda_ok):
    """A NaN key makes the heads that see it NaN, an infinite score of +inf too; a value of
    inf shows in the output; other key heads and rows are untouched."""
    q, k, v, table, lengths = setup([100, 100, 100, 100], 4, 2, 64, 16)
    base = torch.empty_like(q)
    sk.decode_attention_bf16(q, k, v, table, lengths, base)
    k, v = k.clone(), v.clone()
    k[table[0, 2].long(), 3, 0] = float("nan")
    q[1, 2:] = q[1, 2:].abs()
    k[table[1, 0].long(), 0, 1] = float("inf")
    v[table[2, 6].long(), 3, 0, 5] = float("inf")
    out = torch.empty_like(q)
    sk.decode_attention_bf16(q, k, v, table, lengths, out)
    assert torch.isnan(out[0, :2]).all() and torch.equal(out[0, 2:], base[0, 2:])
    assert torch.isnan(out[1, 2:]).all() and torch.equal(out[1, :2], base[1, :2])
    assert torch.isinf(out[2, :2, 5]).all() and torch.equal(out[2, 2:], base[2, 2:])
    assert torch.equal(out[2, :2, :5], base[2, :2, :5])
    assert torch.equal(out[3], base[3])


def test_scores_far_apart(cuda_ok):
    """Scores from very negative to very positive, the maximum growing along the row: the
    running maximum is corrected at every step."""
    D, n = 64, 700
    q, k, v, table, lengths = setup([n], 8, 1, D, 16)
    q.fill_(1.0)
    flat = torch.arange(n, device="cuda")
    at = table[0].long()[flat // 16]
    k[at, flat % 16, 0] = ((flat.float() - n / 2) / 40)[:, None].to(torch.bfloat16).expand(n, D)
    run_and_check(q, k, v, table, lengths, scale=1.0)
    run_and_check(q, k, v, table, lengths, scale=-1.0)


def test_drafted_tokens_share_pages(cuda_ok):
    """Four drafted tokens of one sequence: rows with the same table, growing lengths."""
    q, k, v, table, _ = setup([500] * 4, 14, 2, 128, 16)
    table = table[:1].expand(4, -1)
    run_and_check(q, k, v, table.contiguous(), ints([497, 498, 499, 500]))


def test_table_rows_may_be_padded(cuda_ok):
    q, k, v, table, lengths = setup([90, 33], 4, 1, 64, 16)
    wide = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    a, _ = run_and_check(q, k, v, wide[:, :table.shape[1]], lengths)
    b, _ = run_and_check(q, k, v, wide, lengths)
    assert torch.equal(a, b)


def test_offsets_past_32_bits(cuda_ok):
    """Pages 2^31 elements apart: the last one starts 8 GB into the pool."""
    D, page, step = 64, 64, (1 << 31) + 64
    pool = torch.empty(2 * step + 4 * page * D, dtype=torch.bfloat16, device="cuda")
    k = pool.as_strided((3, page, 1, D), (step, D, D, 1))
    v = pool.as_strided((3, page, 1, D), (step, D, D, 1), storage_offset=2 * page * D)
    for t in (k, v):
        t.copy_(torch.randn(3, page, 1, D, device="cuda"))
    q = torch.randn(2, 4, D, device="cuda").to(torch.bfloat16)
    run_and_check(q, k, v, ints([[2, 0, 1], [1, 2, 0]]), ints([150, 192]))


def test_offsets_past_36_bits(cuda_ok):
    """Pages 2^34 + 64 elements apart: the pool spans more than 2^32 chunks of 16 bytes, which
    the kernel's short addresses do not reach."""
    D, page, step = 128, 16, (1 << 34) + 64
    free, _ = torch.cuda.mem_get_info()
    if free < (80 << 30):
        pytest.skip("needs 80 GB of free memory")
    pool = torch.empty(2 * step + 4 * page * D, dtype=torch.bfloat16, device="cuda")
    k = pool.as_strided((3, page, 1, D), (step, D, D, 1))
    v = pool.as_strided((3, page, 1, D), (step, D, D, 1), storage_offset=2 * page * D)
    for t in (k, v):
        t.copy_(torch.randn(3, page, 1, D, device="cuda"))
    for heads in (4, 12):
        q = torch.randn(2, heads, D, device="cuda").to(torch.bfloat16)
        run_and_check(q, k, v, ints([[2, 0, 1], [1, 2, 0]]), ints([48, 37]))
    del pool, k, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("Hq,Hkv,D", [(1024, 1024, 64), (1024, 8, 64), (512, 512, 128)])
def test_most_heads(cuda_ok, Hq, Hkv, D):
    run_and_check(*setup([33, 70], Hq, Hkv, D, 16, seed=Hq))


def test_given_stream(cuda_ok):
    """The stream argument, with the calling thread's current stream another one."""
    args = setup([3000, 40], 8, 2, 128, 16)
    want, _ = run_and_check(*args)
    st = torch.cuda.Stream()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    sk.decode_attention_bf16(*args, out, stream=st)
    st.synchronize()
    assert torch.equal(out, want)


def test_same_bits_every_time_and_workspace_left_zeroed(cuda_ok):
    ws = sk.attention_workspace()
    args = setup([30000, 5, 800], 16, 2, 128, 32)
    first, _ = run_and_check(*args, workspace=ws)
    counters = ws[:4 * 2 * torch.cuda.get_device_properties(0).multi_processor_count * 4]
    for _ in range(20):
        out = torch.empty_like(first)
        sk.decode_attention_bf16(*args, out, workspace=ws)
        assert torch.equal(out, first)
        assert not counters.any()


def test_workspace_too_small_is_refused(cuda_ok):
    q, k, v, table, lengths = setup([10], 4, 1, 64, 16)
    ws = sk.attention_workspace()[:-16]
    with pytest.raises(sk.SkinnyError) as e:
        sk.decode_attention_bf16(q, k, v, table, lengths, torch.empty_like(q), workspace=ws)
    assert e.value.status == 2


def test_host_tensors_are_refused(cuda_ok):
    q, k, v, table, lengths = setup([10], 4, 1, 64, 16)
    with pytest.raises(TypeError):
        sk.decode_attention_bf16(q, k, v, table.cpu(), lengths, torch.empty_like(q))
    with pytest.raises(TypeError):
        sk.decode_attention_bf16(q, k, v, table, lengths.long(), torch.empty_like(q))


def test_two_streams_at_once(cuda_ok):
    """Calls without a workspace on two streams: one each, results as alone."""
    sets = [setup([20000, 3000], 8, 1, 128, 16, seed=s) for s in (1, 2)]
    want = []
    for s in sets:
        out = torch.empty_like(s[0])
        sk.decode_attention_bf16(*s, out)
        want.append(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(s[0]) for s in sets]
    for _ in range(30):
        for st, s, o in zip(streams, sets, outs):
            with torch.cuda.stream(st):
                sk.decode_attention_bf16(*s, o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("pdl", [False, True])
def test_graphs_replayed_side_by_side_and_with_new_lengths(cuda_ok, pdl):
    """Two graphs captured without a workspace and replayed on two streams; then the
    lengths change in place and a replay follows them."""
    sets = [setup([9000, 400], 8, 1, 128, 16, seed=s) for s in (3, 4)]
    want, graphs, outs = [], [], []
    for s in sets:
        out = torch.empty_like(s[0])
        sk.decode_attention_bf16(*s, out, pdl=pdl)
        torch.cuda.synchronize()
        want.append(out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sk.decode_attention_bf16(*s, out, pdl=pdl)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    q, k, v, table, lengths = sets[0]
    lengths.copy_(ints([17, 8999]).clamp(max=9000))
    graphs[0].replay()
    torch.cuda.synchronize()
    ref, _, tol, _ = attention_reference(q, k, v, table, lengths, 128 ** -0.5)
    check_close(outs[0], ref, tol, "out")


def test_random_cases(cuda_ok):
    """24 seeded random problems over the whole accepted range."""
    import random
    r = random.Random(20261206)
    for i in range(24):
        D = r.choice([64, 96, 128, 192, 256])
        Hkv = r.choice([1, 2, 3, 8])
        G = r.choice([1, 2, 5, 8, 9, 16, 17, 32, 48])
        R = r.choice([1, 2, 7, 33])
        top = r.choice([1, 40, 700, 6000])
        lengths = [r.randint(0, top) for _ in range(R)]
        lengths[0] = top
        window = r.choice([0, 0, 1, 50, 1000])
        run_and_check(*setup(lengths, G * Hkv, Hkv, D, r.choice([1, 7, 16, 64]),
                             r.choice(["nhd", "hnd", "kv", "padded"]), seed=i),
                      window=window, sinks=r.choice([0, 1, 30]))
