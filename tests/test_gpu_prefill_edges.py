"""Prefill where it can go wrong: values that are not finite in slots that a row does not see,
scores at the ends of their range, bad pages and lengths, long caches, captured calls, workspaces."""
import math
import random

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import bits, make_cache, make_table, nan_bits
from tests.test_gpu_prefill import check, prefill64, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()


def _offsets(new):
    return [sum(new[:i]) for i in range(len(new) + 1)]


def _seen(lens, new, b, j, window):
    """Rows of the call that see key j of sequence b."""
    first = sum(new[:b])
    pos = [lens[b] - new[b] + i for i in range(new[b])]
    return [first + i for i, p in enumerate(pos)
            if j <= p and (window < 0 or j >= p - window)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [-1, 50])
@pytest.mark.parametrize("d,heads,group,new,lens", [
    ((128, 128), 2, 4, [70, 5], [300, 133]), ((64, 64), 1, 1, [300], [300]),
    ((192, 128), 1, 8, [3, 40], [130, 40])])
@pytest.mark.parametrize("side", ["k", "v"])
def test_not_finite_only_where_seen(kind, window, d, heads, group, new, lens, side):
    """One key's (or value's) row of NaN or infinities: rows that see it come out not finite, the
    others as if it were any other."""
    page = 16
    cache, q, kc, vc, ks, vs, table, lens_d = setup(1, heads, group, *d, page, kind, "token", new,
                                                    lens, window)
    scale = 1.0 / math.sqrt(d[0])
    cu = _offsets(new)
    want = prefill64(q, kc, vc, table, lens, new, page, scale, window, ks, vs)
    for b in range(len(new)):
        for j in (lens[b] - 1, lens[b] - new[b] // 2 - 1, lens[b] - new[b], 1):
            c = kc if side == "k" else vc
            at = (int(table[b, j // page]), j % page)
            keep = bits(c)[at].clone()
            if kind == "bf16" and j % 2:
                bits(c)[at] = torch.tensor([0x7F80, -0x80], dtype=torch.int16).cuda().repeat(
                    c.shape[3] // 2)  # infinities of both signs
            else:
                bits(c)[at][:, 3] = nan_bits(c)
            o, lse = binding.prefill(cache, q, table, lens_d, window_left=window, cu_seqlens=cu)
            bits(c)[at] = keep
            seen = torch.zeros(sum(new), dtype=torch.bool)
            seen[_seen(lens, new, b, j, window)] = True
            assert torch.isfinite(o[~seen]).all()
            check((o[~seen], lse[~seen]), [t[~seen] for t in want], f"key {j}")
            fine = torch.isfinite(o.float()).all(-1)
            assert not fine[seen].any() or (side == "k" and kind == "bf16" and j % 2)
    assert binding.attn_cache_status() == binding.ATTN_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("size", [1e3, 1e8, 1e15])
@pytest.mark.parametrize("new,lens", [([9], [400]), ([150], [290])])
def test_large_finite_scores(kind, size, new, lens):
    """Scores far apart: the largest key of each row takes all the weight, whatever their size."""
    heads, group, page, d = 1, 2, 16, 64
    cache, q, kc, vc, ks, vs, table, lens_d = setup(2, heads, group, d, d, page, kind, "token", new,
                                                    lens)
    q = (q.float() * size).to(torch.bfloat16)
    got = binding.prefill(cache, q, table, lens_d, scale=0.125)
    ref = prefill64(q, kc, vc, table, lens, new, page, 0.125, -1, ks, vs)
    # rows whose best two scores are further apart than twice the error of a score
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
    sure = ref[2].amax(-1) < 0.05
    if size > 1e7:
        # bounds of scores no longer say anything: the largest key's value alone is left
        pos = torch.arange(lens[0] - new[0], lens[0], device="cuda")
        j = torch.arange(lens[0], device="cuda")
        at = (table[0].long()[j // page], j % page)
        k, v = (bits(c)[at].view(c.dtype).double()[:, 0] for c in (kc, vc))
        if ks is not None:
            k, v = k * ks.double(), v * vs.double()
        x = (q.double() @ k.T).masked_fill(j > pos[:, None, None], -math.inf)
        top = x.topk(2, -1)
        gap = (top.values[..., 0] - top.values[..., 1]) / top.values.abs().amax(-1)
        sure = gap > 1e-4  # (an fp32 score is off by 2^-17 of its terms' sum at most)
        assert sure.float().mean() > 0.8
        want = v[top.indices[..., 0]]
        # one bf16 rounding of the weight's product and one of O
        assert ((got[0].double() - want).abs() <= 2.0 ** -7 * want.abs())[sure].all()
    else:
        check((got[0][sure], got[1][sure]), [t[sure] for t in ref])


def test_scores_of_minus_infinity():
    heads, group, page, d = 1, 4, 16, 128
    new, lens = [3, 2], [40, 200]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(3, heads, group, d, d, page, "bf16", "token",
                                                    new, lens)
    # a column of -inf in the keys of sequence 0 and a positive query there: all scores -inf
    at = (table[0].long()[torch.arange(40).cuda() // page], torch.arange(40).cuda() % page)
    kc[at] = torch.cat([torch.full((40, 1, 1), -math.inf, device="cuda", dtype=torch.bfloat16),
                        kc[at][..., 1:]], -1)
    q[:, :, 0] = 1.0
    o, lse = binding.prefill(cache, q, table, lens_d, cu_seqlens=_offsets(new))
    assert (o[:3] == 0).all() and (lse[:3] == -math.inf).all()
    assert torch.isfinite(o[3:]).all() and torch.isfinite(lse[3:]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_pages_and_lengths(kind):
    """Tokens of a page outside the cache, and lengths beyond the table, are reported and not
    attended; everything else is as it is."""
    heads, group, page, d = 2, 2, 16, 64
    new, lens = [5, 5, 5], [100, 100, 300]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(4, heads, group, d, d, page, kind, "token", new,
                                                    lens, poison=False)
    good = binding.prefill(cache, q, table, lens_d)
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        broken = table.clone()
        broken[1, 2] = bad  # keys 32 .. 47 of sequence 1
        o, lse = binding.prefill(cache, q, broken, lens_d)
        assert binding.attn_cache_status() == binding.ATTN_ERR_BAD_PAGE
        assert torch.equal(o[:5], good[0][:5]) and torch.equal(o[10:], good[0][10:])
        # sequence 1 without those keys
        short = lens[1] - 16
        j = torch.tensor([i for i in range(100) if not 32 <= i < 48]).cuda()
        at = (table[1].long()[j // page], j % page)
        t2, pages = make_table([short], page, 9)
        k2, v2 = (torch.zeros((pages,) + c.shape[1:], dtype=c.dtype, device="cuda") for c in (kc, vc))
        to = (t2[0].long()[torch.arange(short).cuda() // page], torch.arange(short).cuda() % page)
        for a, b in ((k2, kc), (v2, vc)):
            bits(a)[to] = bits(b)[at]
        ref = prefill64(q[5:10], k2, v2, t2, [short], [5], page, 0.125, -1, ks, vs)
        check((o[5:10], lse[5:10]), ref)
    # lengths past the table's room: its keys alone, which all rows see
    o, lse = binding.prefill(cache, q, table[:, :6].contiguous(), lens_d)
    assert binding.attn_cache_status() == binding.ATTN_ERR_BAD_PAGE
    assert torch.isfinite(o).all() and binding.attn_cache_status() == binding.ATTN_OK
    for length in (-5, 0):
        lens_d[0] = length
        o, lse = binding.prefill(cache, q, table, lens_d)
        assert (o[:5] == 0).all() and (lse[:5] == -math.inf).all()
        assert torch.equal(o[5:], good[0][5:]) or torch.allclose(o[5:].float(), good[0][5:].float(),
                                                                 atol=2e-2)
    assert binding.attn_cache_status() == binding.ATTN_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_beyond_32_bits(kind):
    """Pages whose bytes lie beyond 4 GiB of the cache's base."""
    heads, group, page, d = 4, 2, 64, 128
    pages = 180000 if kind == "e4m3" else 90000  # 5.9 GB a side
    dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    kc, vc = (torch.empty(pages, page, heads, d, dtype=dtype, device="cuda") for _ in range(2))
    lens, new = [200, 70], [20, 70]
    table = torch.tensor([[pages - 1, 3, pages - 77, pages // 2 + 5], [pages - 2, pages - 3, 0, 0]],
                         dtype=torch.int32).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    for c in (kc, vc):
        for p in table.unique().tolist():
            x = torch.randn(page, heads, d, generator=g, device="cuda")
            c[p] = (x * 32).to(dtype) if kind == "e4m3" else x.to(dtype)
    unit = torch.full((heads,), 1 / 64).cuda() if kind == "e4m3" else None
    cache = binding.PagedCache(kc, vc, unit, unit)
    q = torch.randn(90, heads * group, d, generator=g, device="cuda").to(torch.bfloat16)
    got = binding.prefill(cache, q, table, torch.tensor(lens, dtype=torch.int32).cuda(),
                          cu_seqlens=_offsets(new))
    ref = prefill64(q, kc, vc, table, lens, new, page, 1 / math.sqrt(d), -1, unit, unit)
    check(got, ref)
    assert binding.attn_cache_status() == binding.ATTN_OK


def test_captured_replayed_and_workspaces():
    """A captured call follows the lengths, tables and queries of each replay; a workspace that
    holds anything, calls of other sizes between, another stream and given outputs."""
    heads, group, page, d = 2, 4, 16, 128
    new = [3, 3, 3, 3]
    most = [500, 900, 64, 300]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(5, heads, group, d, d, page, "bf16", "token",
                                                    new, most, poison=False)
    scale = 1 / math.sqrt(d)
    ws = binding.prefill_workspace()
    ws.fill_(255)
    out = (torch.empty(12, heads * group, d, dtype=torch.bfloat16, device="cuda"),
           torch.empty(12, heads * group, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.prefill(cache, q, table, lens_d, workspace=ws, out=out, stream=side)
    side.synchronize()
    assert got[0] is out[0] and got[1] is out[1]
    check(out, prefill64(q, kc, vc, table, most, new, page, scale))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.prefill(cache, q, table, lens_d, workspace=ws, out=out)
    for lens in ([3, 900, 0, 200], [500, 4, 64, 2], [130, 131, 63, 257]):
        lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, device="cuda").to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        check(out, prefill64(q, kc, vc, table, lens, new, page, scale), str(lens))
        alone = binding.prefill(cache, q, table, lens_d)
        assert torch.equal(alone[0], out[0]) and torch.equal(alone[1], out[1])
    o, none = binding.prefill(cache, q, table, lens_d, with_lse=False, workspace=ws)
    assert none is None and torch.equal(o, out[0])
    assert binding.attn_cache_status() == binding.ATTN_OK


def test_strided_queries_and_empty_calls():
    heads, group, page, d = 2, 3, 8, 64
    new, lens = [7, 9], [70, 9]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(6, heads, group, d, d, page, "bf16", "joint",
                                                    new, lens)
    wide = torch.randn(16, heads * group + 5, d, device="cuda").to(torch.bfloat16)
    wide[:, 2:2 + heads * group] = q
    view = wide[:, 2:2 + heads * group]
    a = binding.prefill(cache, view, table, lens_d, cu_seqlens=_offsets(new))
    b = binding.prefill(cache, q, table, lens_d, cu_seqlens=_offsets(new))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    o, lse = binding.prefill(cache, q[:0], table, lens_d, cu_seqlens=[0, 0, 0])
    assert o.shape == (0, 6, 64) and lse.shape == (0, 6)
    o, lse = binding.prefill(cache, q[:0], table[:0], lens_d[:0])
    assert o.shape == (0, 6, 64)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 40, 10 ** 6])
def test_windows_longer_than_anything(window):
    heads, group, page, d = 1, 2, 16, 64
    new, lens = [20], [333]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(7, heads, group, d, d, page, "bf16", "token",
                                                    new, lens)
    a = binding.prefill(cache, q, table, lens_d, window_left=window)
    b = binding.prefill(cache, q, table, lens_d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,group,new,lens", [((128, 128), 2, [9], [400]), ((64, 64), 1, [300], [700]),
                                              ((192, 128), 4, [70, 1], [200, 900])])
def test_queries_of_many_sizes(kind, d, group, new, lens):
    """Rows from zero to large, and one element far above the others in a column without keys."""
    heads, page = 2, 16
    cache, q, kc, vc, ks, vs, table, lens_d = setup(3, heads, group, *d, page, kind, "token", new,
                                                    lens, poison=False)
    bits(kc)[..., 5] = 0
    sizes = torch.tensor([0.0, 2.0 ** -133, 2.0 ** -110, 2.0 ** -40, 2.0 ** -3, 1.0, 2.0])
    rows = sum(new) * heads * group
    of = sizes[torch.arange(rows) % len(sizes)].view(sum(new), heads * group, 1).cuda()
    q = (q.float() * of).to(torch.bfloat16)
    for spike in (None, 2.0 ** 16, 3e38):
        if spike is not None:
            q[..., 5] = spike
            if spike > 1e30:  # (the others' exact value no longer counts beside it)
                q[..., :5], q[..., 6:] = 0, 0
        got = binding.prefill(cache, q, table, lens_d, cu_seqlens=_offsets(new))
        check(got, prefill64(q, kc, vc, table, lens, new, page, 1 / math.sqrt(d[0]), -1, ks, vs),
              f"spike {spike}")
    assert binding.attn_cache_status() == binding.ATTN_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_sequences(kind):
    """More units than a CTA has threads, and more sequences than a table of offsets takes."""
    heads, group, page, d = 1, 2, 16, 64
    lens = [1 + 37 * i % 61 for i in range(1500)]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(8, heads, group, d, d, page, kind, "token",
                                                    [1] * 1500, lens)
    got = binding.prefill(cache, q, table, lens_d)
    check(got, prefill64(q, kc, vc, table, lens, [1] * 1500, page, 0.125, -1, ks, vs))
    assert binding.attn_cache_status() == binding.ATTN_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [(64, 64), (128, 128), (192, 128)])
def test_short_and_long_chunks_in_turn(kind, d):
    """Units of one query tile and of two behind each other on every SM, with one key tile or more."""
    heads, group, page = 2, 4, 64
    rng = random.Random(5)
    new = [rng.choice([1, 1, 3, 40, 64, 33, 2]) for _ in range(450)]
    lens = [n + rng.choice([0, 5, 100, 130, 300, 517]) for n in new]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(11, heads, group, *d, page, kind, "token", new,
                                                    lens)
    ref = prefill64(q, kc, vc, table, lens, new, page, 1 / math.sqrt(d[0]), -1, ks, vs)
    for _ in range(3):
        got = binding.prefill(cache, q, table, lens_d, cu_seqlens=_offsets(new))
        check(got, ref)
    assert binding.attn_cache_status() == binding.ATTN_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_sides_of_different_orders(kind):
    """Keys token by token and values head by head, pages of 24 tokens."""
    heads, group, page, d = 3, 2, 24, 128
    new, lens = [40, 3], [500, 50]
    table, pages = make_table(lens, page, 1)
    kc = make_cache(pages, page, heads, d, kind, "token", 2)
    vc = make_cache(pages, page, heads, d, kind, "head", 3)
    unit = torch.full((heads,), 1 / 64).cuda() if kind == "e4m3" else None
    q = torch.randn(43, heads * group, d, device="cuda").to(torch.bfloat16)
    lens_d = torch.tensor(lens, dtype=torch.int32).cuda()
    for k, v in ((kc, vc), (vc, kc)):
        got = binding.prefill(binding.PagedCache(k, v, unit, unit), q, table, lens_d,
                              cu_seqlens=_offsets(new))
        check(got, prefill64(q, k, v, table, lens, new, page, 1 / math.sqrt(d), -1, unit, unit))


def test_broadcast_caches():
    """A cache whose pages or heads share memory can be read (maps do not describe it: its tiles come
    by rows)."""
    page, d = 16, 64
    g = torch.Generator().manual_seed(3)
    one = torch.randn(40, page, 1, d, generator=g).to(torch.bfloat16).cuda()
    kc = vc = one.expand(40, page, 3, d)
    table, _ = make_table([300, 41], page, 4)
    lens = [300, 41]
    q = torch.randn(12, 6, d, generator=g).to(torch.bfloat16).cuda()
    got = binding.prefill(binding.PagedCache(kc, vc), q, table,
                          torch.tensor(lens, dtype=torch.int32).cuda())
    dense = one.expand(40, page, 3, d).contiguous()
    check(got, prefill64(q, dense, dense, table, lens, [6, 6], page, 1 / math.sqrt(d)))
