"""attn_decode on the GPU against 64-bit attention over the same cache: head layouts, lengths
from none to long, page sizes, windows, both cache types, bad pages, workspaces, captured
calls.  Every slot that no sequence sees holds NaN."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import (bits, check_decode, decode64, make_cache, make_table, nan_bits,
                                poison_unseen)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ws():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()
    return binding.decode_workspace()


class Case:
    def __init__(self, d, kind, lens, heads, group, page=16, order="token", window=-1, seed=1,
                 scales=True, peak=1.0):
        dqk, dv = d
        self.lens, self.page, self.window = lens, page, window
        self.table, pages = make_table(lens, page, seed)
        self.kc = make_cache(pages, page, heads, dqk, kind, order, seed + 1)
        self.vc = make_cache(pages, page, heads, dv, kind, order, seed + 2)
        poison_unseen(self.kc, self.table, lens, page, window)
        poison_unseen(self.vc, self.table, lens, page, window)
        g = torch.Generator(device="cpu").manual_seed(seed + 3)
        e = kind == "e4m3" and scales
        unit = lambda: (torch.rand(heads, generator=g) / 40 + 0.01).cuda()
        self.ks, self.vs = (unit(), unit()) if e else (None, None)
        if kind == "e4m3" and not scales:
            peak = peak / 40
        # queries as a slice of a wider row
        row = torch.randn(len(lens), heads * group * dqk + 64, generator=g)
        self.q = (row * peak).to(torch.bfloat16).cuda()[:, :heads * group * dqk].unflatten(
            1, (heads * group, dqk))
        self.scale = 1.0 / math.sqrt(dqk)
        self.cache = binding.PagedCache(self.kc, self.vc, self.ks, self.vs)
        self.lens_t = torch.tensor(lens, dtype=torch.int32).cuda()

    def run(self, ws, **kw):
        return binding.decode(self.cache, self.q, self.table, self.lens_t, scale=self.scale,
                              window_left=self.window, workspace=ws, **kw)

    def ref(self, **kw):
        return decode64(self.q, self.kc, self.vc, self.table, self.lens, self.page, self.scale,
                        self.window, self.ks, self.vs, **kw)

    def check(self, ws):
        got = self.run(ws)
        check_decode(got, self.ref())
        assert binding.attn_cache_status() == binding.ATTN_OK
        return got


RAGGED = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 300]


@pytest.mark.parametrize("d", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,group", [(1, 1), (3, 2), (2, 8), (2, 9), (1, 16), (2, 17),
                                         (1, 24), (1, 32), (1, 40), (1, 71)])
def test_heads_and_lengths(ws, d, kind, heads, group):
    Case(d, kind, RAGGED, heads, group).check(ws)


@pytest.mark.parametrize("d", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,order", [(1, "token"), (7, "token"), (16, "head"), (24, "joint"),
                                        (64, "joint"), (128, "head"), (1000, "token")])
def test_pages_and_layouts(ws, d, kind, page, order):
    Case(d, kind, [500, 1, 0, 77, 1000], 2, 4, page=page, order=order, scales=False).check(ws)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 1, 15, 16, 63, 64, 100, 5000])
def test_windows(ws, kind, window):
    Case((128, 128), kind, [1, 16, 17, 64, 100, 333, 1000, 0], 2, 3, page=24,
         window=window).check(ws)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,group,n", [(1, 1, 20011), (1, 8, 70001), (2, 12, 40000),
                                           (1, 32, 9000), (16, 1, 5000)])
def test_long_sequences_are_joined(ws, kind, heads, group, n):
    """One sequence shared by up to all CTAs: one level of joining and two."""
    Case((128, 128), kind, [n], heads, group, page=64, peak=2.0).check(ws)


def test_long_and_short_together(ws):
    Case((64, 64), "bf16", [30000] + [5] * 40 + [0] * 3 + [4000], 2, 4, page=32).check(ws)


@pytest.mark.parametrize("kind,lens", [("bf16", [70001, 64000, 60007, 66000]),
                                       ("e4m3", [140001, 128000, 120007, 132000])])
def test_claimed_pieces(ws, kind, lens):
    """A line long enough that its CTAs claim pieces of it: right, the same bits every time
    (whichever CTA works on a piece), and the claims are back at zero for the next call."""
    c = Case((64, 64), kind, lens, 8, 2, page=64)
    small = Case((64, 64), kind, [100, 0, 3000], 8, 2, page=64)
    other = small.run(ws)
    first = c.check(ws)
    for _ in range(5):
        got = c.run(ws)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
        got = small.run(ws)
        assert torch.equal(got[0], other[0]) and torch.equal(got[1], other[1])


def test_many_sequences(ws):
    """More sequences than a block has threads, and than CTAs."""
    lens = [(i * 37) % 90 for i in range(700)]
    Case((64, 64), "bf16", lens, 1, 2, page=16).check(ws)


def test_peaked_scores(ws):
    """Scores of some hundred: one key has nearly all of the weight, wherever it lies."""
    for seed in range(4):
        Case((128, 128), "bf16", [3000, 700], 2, 8, page=16, peak=40.0, seed=seed).check(ws)


def test_no_lse_given_outputs_and_own_workspace(ws):
    c = Case((128, 128), "bf16", [100, 0, 900], 2, 4)
    o, lse = c.run(ws)
    o2, none = c.run(ws, with_lse=False)
    assert none is None and torch.equal(o, o2)
    out = (torch.zeros_like(o), torch.zeros_like(lse))
    assert c.run(ws, out=out)[0] is out[0]
    assert torch.equal(out[0], o) and torch.equal(out[1], lse)
    o3, lse3 = c.run(None)
    assert torch.equal(o3, o) and torch.equal(lse3, lse)


def test_the_same_bits_again(ws):
    """Parts are joined in their order: no run differs from another, in any workspace."""
    c = Case((128, 128), "bf16", [9000, 50, 0, 3000], 2, 8, page=64)
    first = c.run(ws)
    other = binding.decode_workspace()
    for i in range(20):
        got = c.run(other if i % 2 else ws)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_workspace_serves_calls_of_any_size(ws):
    cases = [Case((128, 128), "bf16", [20000], 1, 16, page=64),
             Case((64, 64), "e4m3", [1, 2, 3], 12, 1),
             Case((192, 128), "bf16", [4000] * 9, 4, 1, page=32),
             Case((128, 128), "e4m3", [300] * 50, 8, 5)]
    want = [c.run(ws) for c in cases]
    for _ in range(3):
        for c, w in zip(cases, want):
            got = c.run(ws)
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    for c, w in zip(cases, want):
        check_decode(w, c.ref())


def test_workspace_without_initialisation():
    c = Case((64, 64), "bf16", [100, 30], 2, 2)
    ws = torch.zeros(binding.attn_decode_workspace_size(), dtype=torch.uint8, device="cuda")
    out = (torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"),
           torch.full((2, 4), 7.0, device="cuda"))
    c.run(ws, out=out)
    assert binding.attn_cache_status() == binding.ATTN_ERR_WORKSPACE_NOT_READY
    assert (out[0] == 7).all() and (out[1] == 7).all()
    assert binding.attn_decode_workspace_init(ws, ws.numel()) == binding.ATTN_OK
    check_decode(c.run(ws, out=out), c.ref())
    assert binding.attn_cache_status() == binding.ATTN_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, "pages"])
def test_bad_pages_take_no_part(ws, kind, bad):
    c = Case((128, 128), kind, [100, 50, 40], 2, 4, page=16)
    c.table[0, 2] = c.kc.shape[0] if bad == "pages" else bad
    c.table[1, 0] = c.table[0, 2]
    c.table[1, 1:] = c.table[0, 2]
    got = c.run(ws)
    assert binding.attn_cache_status() == binding.ATTN_ERR_BAD_PAGE
    assert binding.attn_cache_status() == binding.ATTN_OK
    check_decode(got, c.ref(hidden={0: range(32, 48), 1: range(50)}))


@pytest.mark.parametrize("over", [1, 1000, 2 ** 31 - 1])
def test_length_past_the_table(ws, over):
    c = Case((128, 128), "bf16", [64, 50], 2, 4, page=16)
    room = c.table.shape[1] * 16
    c.lens_t[0] = min(room + over, 2 ** 31 - 1)
    got = c.run(ws)
    assert binding.attn_cache_status() == binding.ATTN_ERR_BAD_PAGE
    check_decode(got, c.ref())  # the keys that the table has
    c.lens_t[0] = -3            # no token: an unused row
    c.lens[0] = 0
    check_decode(c.run(ws), c.ref())
    assert binding.attn_cache_status() == binding.ATTN_OK


def test_values_that_are_not_finite_stay_in_their_row(ws):
    c = Case((128, 128), "bf16", [100, 100], 2, 2, page=16)
    at = (c.table[0, 3].long(), 5)
    bits(c.vc)[at][0, 3] = nan_bits(c.vc)  # a key that sequence 0 sees, key head 0, column 3
    o, lse = c.run(ws)
    assert torch.isnan(o[0, :2, 3]).all() and torch.isfinite(lse).all()
    o[0, :2, 3] = 0
    assert torch.isfinite(o).all()
    bits(c.kc)[at][1, 0] = nan_bits(c.kc)  # key head 1
    o, lse = c.run(ws)
    assert torch.isnan(lse[0, 2:]).all() and torch.isfinite(lse[0, :2]).all()
    assert torch.isnan(o[0, 2:]).all() and torch.isfinite(o[1]).all()


@pytest.mark.parametrize("q_exp,k_exp,v_exp", [(None, -100, 100), (None, 0, 0), (-100, 100, -100),
                                               (60, -60, 0), (-60, 60, 0), (-100, -100, 0)])
def test_e4m3_scales_from_one_end_to_the_other(ws, q_exp, k_exp, v_exp):
    """Queries of zero (None) and of extreme sizes; products of all factors from 2^-200 on."""
    c = Case((128, 128), "e4m3", [20, 1, 700], 2, 4, page=16, scales=False)
    c.q = c.q * 2.0 ** q_exp if q_exp is not None else torch.zeros_like(c.q)
    c.ks, c.vs = torch.full((2,), 2.0 ** k_exp).cuda(), torch.full((2,), 2.0 ** v_exp).cuda()
    c.cache = binding.PagedCache(c.kc, c.vc, c.ks, c.vs)
    c.check(ws)


def test_scores_of_minus_infinity_are_an_empty_row(ws):
    c = Case((64, 64), "bf16", [20, 20], 1, 2, page=16)
    c.kc[c.table[0].long()] = 0
    c.kc[c.table[0].long(), :, :, 0] = -float("inf")
    c.q[0] = 1.0
    o, lse = c.run(ws)
    assert (o[0] == 0).all() and (lse[0] == -math.inf).all() and torch.isfinite(o[1]).all()


@pytest.mark.parametrize("kind,size", [("bf16", 2 ** 31), ("e4m3", 2 ** 32)])
def test_a_cache_beyond_32_bit_offsets(ws, kind, size):
    page, heads, d = 64, 2, 128
    pages = size // (page * heads * d) + 9
    dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    kc = torch.zeros(pages, page, heads, d, dtype=torch.int16 if kind == "bf16" else torch.uint8,
                     device="cuda").view(dtype)
    vc = torch.zeros(kc.shape, dtype=torch.int16 if kind == "bf16" else torch.uint8,
                     device="cuda").view(dtype)
    ids = [pages - 1, 3, pages - 5]
    for t, seed in ((kc, 1), (vc, 2)):
        bits(t)[torch.tensor(ids).cuda()] = bits(make_cache(3, page, heads, d, kind, "token", seed))
    table = torch.tensor([ids], dtype=torch.int32).cuda()
    lens = [150]
    scale = 1.0 / math.sqrt(d) / (1 if kind == "bf16" else 40)
    g = torch.Generator(device="cpu").manual_seed(3)
    q = torch.randn(1, 8, d, generator=g).to(torch.bfloat16).cuda()
    got = binding.decode(binding.PagedCache(kc, vc), q, table,
                         torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale, workspace=ws)
    check_decode(got, decode64(q, kc, vc, table, lens, page, scale))


def test_another_stream(ws):
    c = Case((128, 128), "bf16", [2000, 100], 2, 4, page=64)
    want = c.run(ws)
    s = torch.cuda.Stream()
    own = binding.decode_workspace(stream=s)
    s.wait_stream(torch.cuda.current_stream())
    got = [c.run(own, stream=s) for _ in range(3)]
    got.append(c.run(own, stream=s.cuda_stream))
    s.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_sequences_share_pages(ws, kind):
    """A prompt in common: the same pages in several rows of the table, and twice in one."""
    c = Case((128, 128), kind, [500, 500, 470, 512], 2, 4, page=32)
    c.lens = [500, 490, 470, 512]  # (each sees slots that Case left readable)
    c.lens_t = torch.tensor(c.lens, dtype=torch.int32).cuda()
    c.table[1] = c.table[0]
    c.table[2, :14] = c.table[0, :14]
    c.table[3, 5] = c.table[3, 4]
    c.check(ws)


@pytest.mark.parametrize("window", [-1, 0, 100])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_no_sequence_has_a_key(ws, kind, window):
    """A batch of unused rows alone: zeros, and nothing read through a table of -1."""
    c = Case((128, 128), kind, [0] * 6, 2, 4, page=16, window=window)
    c.lens_t = torch.tensor([0, -1, -2 ** 31, 0, -7, -2 ** 31 + 1], dtype=torch.int32).cuda()
    o, lse = c.check(ws)
    assert (o == 0).all() and (lse == -math.inf).all()


def test_whole_parts_of_minus_infinity(ws):
    """Scores of -inf over the first half of a sequence that many CTAs share."""
    n, hidden = 20000, 10007
    c = Case((128, 128), "bf16", [n], 1, 8, page=16)
    c.q[:, :, 0] = 1.0
    for j in range(hidden // 16 + 1):
        c.kc[int(c.table[0, j]), :min(16, hidden - 16 * j), :, 0] = -float("inf")
    check_decode(c.run(ws), c.ref(hidden={0: range(hidden)}))


def test_two_calls_at_once(ws):
    """Calls on two streams with a workspace each."""
    a = Case((128, 128), "bf16", [9000], 2, 8, page=64, seed=1)
    b = Case((128, 128), "bf16", [7000, 10], 2, 8, page=64, seed=9)
    want = a.run(ws), b.run(ws)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    spaces = [binding.decode_workspace(stream=s) for s in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for c, s, w in zip((a, b), streams, spaces):
            got.append(c.run(w, stream=s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], want[i % 2][0]) and torch.equal(g[1], want[i % 2][1])


def test_captured_calls_share_a_workspace_and_follow_lengths():
    """Two graphs and eager calls on one workspace, one after the other; the captured launch
    takes the lengths that it finds on the device."""
    ws = binding.decode_workspace()
    c = Case((128, 128), "bf16", [4000, 37, 900], 2, 8, page=16)
    small = Case((64, 64), "bf16", [3, 500], 4, 1)
    out = c.run(ws)
    out2 = small.run(ws)
    out, out2 = tuple(t.clone() for t in out), tuple(t.clone() for t in out2)
    graphs = []
    for case, dst in ((c, out), (small, out2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            case.run(ws, out=dst)
        graphs.append(g)
    for lens in ([4000, 37, 900], [1, 0, 2], [3999, 30, 64]):
        c.lens = lens
        c.lens_t.copy_(torch.tensor(lens, dtype=torch.int32))
        for _ in range(2):
            graphs[0].replay()
            graphs[1].replay()
            eager = c.run(ws)
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
        check_decode(out, c.ref())
        check_decode(out2, small.ref())
