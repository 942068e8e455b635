"""decode_attention_shared_prefix_bf16 against a plain implementation in 64 bits."""
import math

import pytest
import torch

import skinny_bf16_gemm_gb300 as sk
from attention_helpers import F64, HALF_BF16, U32, check_close, make_cache

pytestmark = pytest.mark.gpu


def reference(q, k_cache, v_cache, prefix_table, prefix, table, lengths, scale):
    """(out, lse, out_tol, lse_tol) in 64 bits. As for decode_attention_bf16 (scores,
    exponential, sums; at most 256 partials more to join), and the prefix's weights are rounded
    to BF16 in the product with the values and not in their sum: at most half a step of each,
    HALF_BF16 sum_prefix w |v|."""
    R, Hq, D = q.shape
    Hkv, page = k_cache.shape[2], k_cache.shape[1]
    G = Hq // Hkv
    out = torch.zeros(R, Hq, D, dtype=F64, device=q.device)
    lse = torch.full((R, Hq), -math.inf, dtype=F64, device=q.device)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    j = torch.arange(prefix, device=q.device)
    kp, vp = (c[prefix_table.long()[j // page], j % page].to(F64) for c in (k_cache, v_cache))  # [P, Hkv, D]
    for r, n in enumerate(lengths.tolist()):
        j = torch.arange(n, device=q.device)
        at, off = table[r].long()[j // page], j % page
        k, v = torch.cat([kp, k_cache[at, off].to(F64)]), torch.cat([vp, v_cache[at, off].to(F64)])
        if k.shape[0] == 0:
            continue
        qr = q[r].to(F64).view(Hkv, G, D)
        s = torch.einsum("hgd,nhd->hgn", qr, k) * scale
        mag = torch.einsum("hgd,nhd->hgn", qr.abs(), k.abs()) * abs(scale)
        ds = 2 * (D + 2) * U32 * mag.amax(-1) + 4 * U32 * s.abs().amax(-1) + 2.0 ** -21
        steps = 2 * U32 * (k.shape[0] / 16 + 580)
        w = torch.softmax(s, -1)
        out[r] = torch.einsum("hgn,nhd->hgd", w, v).reshape(Hq, D)
        lse[r] = torch.logsumexp(s, -1).reshape(Hq)
        vmax = v.abs().amax(0)[:, None, :]
        tol = 2 * (ds[..., None] + 2.0 ** -15 + steps) * vmax
        tol = tol + HALF_BF16 * torch.einsum("hgn,nhd->hgd", w[..., :prefix], vp.abs())
        out_tol[r] = tol.reshape(Hq, D)
        out_tol[r] += HALF_BF16 * (out[r].abs() + out_tol[r])
        lse_tol[r] = (ds + steps).reshape(Hq) + 4 * U32 * (1 + lse[r].abs())
    return out, lse, out_tol, lse_tol


class Case:
    """Queries, a pool whose pages are dealt out in any order, tables and lengths."""

    def __init__(self, R, Hq, Hkv, D, page, prefix, lengths, layout="nhd", seed=1, q_pad=0, spare=0, wide=True):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        if isinstance(lengths, int):
            lengths = [max(0, (lengths * (7 * r + 3)) % (lengths + 1)) for r in range(R)]
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.prefix = prefix
        width, shared = max(1, -(-max(lengths) // page)) + spare, max(1, -(-prefix // page)) + spare
        pages = shared + R * width
        self.k, self.v = make_cache(pages, page, Hkv, D, layout, seed)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.prefix_table = order[:shared].clone()
        if wide:  # a table of so many tokens that the prefix is read once and joined (but for one row)
            more = -(-((16 << 20) + R * Hq * (20 << 10)) // (R * Hkv * D * 4 * page)) + 1
            self.prefix_table = torch.cat([self.prefix_table, torch.full_like(order[:1], -7).expand(more)])
        self.table = order[shared:].view(R, width).clone()
        self.prefix_length = torch.tensor([prefix], dtype=torch.int32, device="cuda")
        wide = torch.randn(R, Hq * D + q_pad, generator=g, device="cuda").mul_(1.3).to(torch.bfloat16)
        self.q = wide[:, :Hq * D].view(R, Hq, D)
        self.scale = D ** -0.5
        self.out = torch.full((R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((R, Hq), 7.0, device="cuda")

    def call(self, **kw):
        return sk.decode_attention_shared_prefix_bf16(
            self.q, self.k, self.v, self.prefix_table, self.prefix_length, self.table, self.lengths, self.out,
            **dict(dict(scale=self.scale, lse=self.lse), **kw))

    def check(self, **kw):
        assert self.call(**kw) is self.out
        assert sk.device_error() == (0, 0)
        out, lse, out_tol, lse_tol = reference(self.q, self.k, self.v, self.prefix_table, self.prefix, self.table,
                                               self.lengths, self.scale)
        check_close(self.out, out, out_tol, "out")
        check_close(self.lse, lse, lse_tol, "lse")
        return self


# One tile of query rows, two, two with the second partly filled, several blocks; every head
# width; prefixes from one token to many tiles, ending within tiles and pages.
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("R,Hq,Hkv,page,prefix,own", [
    (1, 1, 1, 16, 1, 1), (1, 7, 1, 16, 128, 5), (4, 7, 1, 16, 509, 64), (3, 8, 8, 1, 65, 3), (16, 8, 1, 24, 700, 33),
    (17, 8, 1, 64, 1000, 100), (64, 7, 1, 16, 3001, 200), (5, 12, 4, 8, 4096, 9), (33, 32, 2, 32, 2050, 40),
    (130, 4, 2, 128, 129, 70), (1, 96, 2, 16, 700, 20)])
def test_shapes(cuda_ok, D, R, Hq, Hkv, page, prefix, own, wide):
    Case(R, Hq, Hkv, D, page, prefix, own, seed=D + R, wide=wide).check()


# Pages that no box of 8 tokens fits, of one token and of more than a tile's.
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [1, 4, 12, 100, 1000])
def test_pages_without_boxes(cuda_ok, D, page):
    for R, prefix in ((3, 1601), (40, 1919)):
        Case(R, 8, 1, D, page, prefix, 30, seed=page).check()


# More blocks of query rows than there are CTAs: they are gone through in several passes.
@pytest.mark.parametrize("R,Hq,Hkv,D,page", [(1024, 64, 1, 64, 16), (700, 64, 1, 128, 4), (520, 128, 2, 192, 16)])
def test_more_blocks_than_ctas(cuda_ok, R, Hq, Hkv, D, page):
    c = Case(R, Hq, Hkv, D, page, 301, 3, seed=20)
    c.call()
    assert sk.device_error() == (0, 0)
    for r in (0, R // 3, R // 2, R - 130, R - 1):  # a few rows of every pass
        at = slice(r, r + 1)
        out, lse, out_tol, lse_tol = reference(c.q[at], c.k, c.v, c.prefix_table, c.prefix, c.table[at], c.lengths[at],
                                               c.scale)
        check_close(c.out[at], out, out_tol, "out")
        check_close(c.lse[at], lse, lse_tol, "lse")


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv", "padded"])
@pytest.mark.parametrize("R,Hq,Hkv,D", [(6, 14, 2, 128), (48, 16, 2, 64)])
def test_layouts_and_strides(cuda_ok, layout, R, Hq, Hkv, D, wide):
    Case(R, Hq, Hkv, D, 16, 1111, 90, layout=layout, seed=5, q_pad=24, spare=2, wide=wide).check()


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("R", [2, 40])
@pytest.mark.parametrize("D", [128, 192])
def test_lengths_of_zero_and_one(cuda_ok, R, D, wide):
    Case(R, 7, 1, D, 16, 300, [0, 1] * (R // 2), seed=1, wide=wide).check()  # rows with the prefix alone
    Case(R, 7, 1, D, 16, 1, [0] * R, seed=2, wide=wide).check()
    c = Case(R, 7, 1, D, 16, 0, [0, 5] * (R // 2), seed=3, wide=wide).check()  # no prefix
    assert (c.out[0] == 0).all() and (c.lse[0] == -math.inf).all()
    c = Case(R, 7, 1, D, 16, 0, [0] * R, seed=4, wide=wide).check()
    assert (c.out == 0).all()


def test_a_long_prefix(cuda_ok):
    Case(24, 56, 8, 128, 32, 20011, 50, seed=7).check()


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.7])
def test_other_scales(cuda_ok, scale):
    for R in (3, 30):
        c = Case(R, 8, 1, 128, 16, 777, 40, seed=8)
        c.scale = scale
        c.check()
        c.prefix_table = c.prefix_table[:49]  # 784 tokens: in one launch
        c.check()


def test_growing_scores(cuda_ok):
    """Keys along the queries, ever larger: the maximum moves and O is rescaled at many steps."""
    for R, D in ((4, 128), (40, 128), (40, 64), (4, 256)):
        c = Case(R, 8, 1, D, 16, 2000, 30, seed=9)
        direction = torch.sign(c.q[0, 0].float())
        j = torch.arange(2000, device="cuda")
        at, off = c.prefix_table.long()[j // 16], j % 16
        c.k[at, off, 0] = (direction[None, :] * (j[:, None] / 400.0)).to(torch.bfloat16)
        c.check()


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("bad", ["prefix page", "own page", "prefix length", "lengths"])
def test_bad_indices_are_reported(cuda_ok, bad, wide):
    for R in (5, 40):
        c = Case(R, 8, 1, 128, 16, 640, 64, seed=10, wide=wide)
        c.lengths[:] = 64
        if bad == "prefix page":
            c.prefix_table[3], c.prefix_table[17] = -1, c.k.shape[0]
        elif bad == "own page":
            c.table[2, 1] = 1 << 30
        elif bad == "prefix length":
            c.prefix_length[0] = 16 * c.prefix_table.numel() + 17
        else:
            c.lengths[1] = -1
        c.call()
        st, word = sk.device_error()
        assert sk.STATUS[st] == "SKINNY_ERR_INDEX" and word == 256
        # As with those tokens left out, or the nearest length.
        got, got_lse = c.out.clone(), c.lse.clone()
        if bad == "prefix page":
            keep = [i for i in range(40) if i not in (3, 17)]  # a table of all the pages that are seen
            c.prefix_table, c.prefix = c.prefix_table[keep].clone(), 640 - 32
        elif bad == "own page":
            c.table[2, 1], c.lengths[2] = c.table[2, 3], 48
        elif bad == "prefix length":
            c.prefix = 640
        else:
            c.lengths[1] = 0
        c.prefix_length[0] = c.prefix
        out, lse, out_tol, lse_tol = reference(c.q, c.k, c.v, c.prefix_table, c.prefix, c.table, c.lengths, c.scale)
        check_close(got, out, out_tol, bad)
        check_close(got_lse, lse, lse_tol, bad)


@pytest.mark.parametrize("wide", [True, False])
def test_infinities_and_nan(cuda_ok, wide):
    for R in (3, 40):
        c = Case(R, 8, 2, 128, 16, 500, 20, seed=11, wide=wide)
        at = c.prefix_table.long()[0]
        c.v[c.prefix_table.long()[2], 3, 0, 5] = math.inf  # value 5 of the first key head's rows
        c.k[at, 1, 1, 0] = math.nan                        # every score of it for the second's
        c.call()
        assert sk.device_error() == (0, 0)
        first, second = c.out[:, :4].float(), c.out[:, 4:]
        assert (first[:, :, 5] == math.inf).all() and torch.isnan(second).all()
        assert torch.isnan(c.lse[:, 4:]).all()
        rest = [i for i in range(128) if i != 5]
        c.v[c.prefix_table.long()[2], 3, 0, 5] = 0.0
        c.k[at, 1, 1, 0] = 0.0
        out, lse, out_tol, lse_tol = reference(c.q, c.k, c.v, c.prefix_table, c.prefix, c.table, c.lengths, c.scale)
        check_close(first[:, :, rest], out[:, :4][:, :, rest], out_tol[:, :4][:, :, rest], "out")
        check_close(c.lse[:, :4], lse[:, :4], lse_tol[:, :4], "lse")


@pytest.mark.parametrize("wide", [True, False])
def test_places_beyond_the_prefix_are_not_read(cuda_ok, wide):
    """NaN in the rest of the last pages, and table entries after them that are no pages."""
    for R in (3, 40):
        c = Case(R, 7, 1, 128, 16, 500, [37] * R, seed=12, spare=3, wide=wide)
        c.prefix_table[32:] = -5
        c.table[:, 3:] = 1 << 29
        for t in (c.k, c.v):
            t[c.prefix_table.long()[31], 4:] = math.nan
            t[c.table[:, 2].long(), 5:] = math.nan
        c.check()


def test_same_bits_again_and_on_another_stream(cuda_ok):
    for R, D in ((4, 128), (64, 128), (64, 64), (9, 256)):
        c = Case(R, 8, 1, D, 16, 5000, 300, seed=13)
        c.call()
        out, lse = c.out.clone(), c.lse.clone()
        s = torch.cuda.Stream()
        for kw in (dict(pdl=True), dict(stream=s), dict(workspace=sk.shared_prefix_workspace(R, 8, 1, D))):
            for _ in range(3):
                c.out.fill_(0)
                torch.cuda.synchronize()
                c.call(**kw)
                torch.cuda.synchronize()
                assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


def test_one_workspace_for_several_sizes(cuda_ok):
    ws = sk.shared_prefix_workspace(64, 16, 2, 128)
    cases = [Case(64, 16, 2, 128, 16, 900, 50, seed=14), Case(3, 8, 1, 64, 16, 200, 5, seed=15),
             Case(40, 16, 2, 128, 16, 130, 600, seed=16)]
    for _ in range(3):
        for c in cases:
            c.check(workspace=ws)


def test_captured_steps_with_growing_lengths(cuda_ok):
    """Two graphs with workspaces of their own, replayed side by side; the lengths grow between
    replays, as in decoding."""
    cases = [Case(32, 8, 1, 128, 16, 2000, [40] * 32, seed=17), Case(6, 8, 1, 128, 16, 3000, [50] * 6, seed=18)]
    graphs = []
    for c in cases:
        c.call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for step in range(4):
        for c in cases:
            c.lengths -= 3
            c.prefix -= 100
            c.prefix_length[0] = c.prefix
            c.out.fill_(0)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c in cases:
            out, lse, out_tol, lse_tol = reference(c.q, c.k, c.v, c.prefix_table, c.prefix, c.table, c.lengths, c.scale)
            check_close(c.out, out, out_tol, "out")
            check_close(c.lse, lse, lse_tol, "lse")


def test_as_decode_attention_over_the_joined_tables(cuda_ok):
    """The two operators on the same tokens: the prefix a whole number of pages."""
    for R, Hq, Hkv, D in ((5, 14, 2, 128), (64, 32, 8, 64)):
        c = Case(R, Hq, Hkv, D, 16, 1600, 100, seed=19)
        c.check()
        table = torch.cat([c.prefix_table[None, :100].expand(R, -1), c.table], 1).contiguous()
        out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
        sk.decode_attention_bf16(c.q, c.k, c.v, table, c.lengths + 1600, out, lse=lse)
        assert (out.float() - c.out.float()).abs().max() < 0.02 and (lse - c.lse).abs().max() < 1e-4


def test_two_streams_at_once(cuda_ok):
    """Every stream has a workspace of its own without one being named."""
    cases = [Case(32, 8, 1, 128, 16, 4000, 500, seed=21), Case(6, 16, 2, 64, 16, 6000, 700, seed=22),
             Case(5, 8, 1, 128, 16, 200, 700, seed=23, wide=False)]
    want = []
    for c in cases:
        c.check()
        want.append((c.out.clone(), c.lse.clone()))
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, c in zip(streams, cases):
            c.call(stream=s)
    torch.cuda.synchronize()
    assert sk.device_error() == (0, 0)
    for c, (out, lse) in zip(cases, want):
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


def test_the_last_page_of_a_pool_past_32_bits(cuda_ok):
    """Element offsets of more than 2^32 (2^33 bytes), by boxes and by single tokens."""
    for page in (64, 12):
        D, pages = 128, (1 << 32) // (page * 128) + 70
        k = torch.empty(pages, page, 1, D, dtype=torch.bfloat16, device="cuda")
        c = Case(20, 8, 1, D, page, 900, 90, seed=24)
        used = c.k.shape[0]
        k[-used:] = c.k  # the keys' pages at the end of a long pool, the values' too
        v = torch.empty_like(k)
        v[-used:] = c.v
        for t in (c.prefix_table, c.table):
            t[t >= 0] += pages - used
        c.k, c.v = k, v
        c.check()
        del k, v, c
        torch.cuda.empty_cache()


def test_a_workspace_too_small_is_refused(cuda_ok):
    for wide in (True, False):
        c = Case(6, 8, 1, 128, 16, 200, 20, seed=25, wide=wide)
        ws = sk.shared_prefix_workspace(6, 8, 1, 128)
        c.check(workspace=ws)
        with pytest.raises(sk.SkinnyError) as e:
            c.call(workspace=ws[:-1])
        assert sk.STATUS[e.value.status] == "SKINNY_ERR_SHAPE"
        with pytest.raises(sk.SkinnyError) as e:
            c.call(workspace=ws.cpu())
        assert sk.STATUS[e.value.status] == "SKINNY_ERR_DEVICE"
