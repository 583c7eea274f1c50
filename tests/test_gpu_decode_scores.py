"""attn_decode over scores and weights at the ends of their ranges."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import (BF16_HALF, bits, check_decode, decode64, make_cache, make_table)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ws():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()
    return binding.decode_workspace()


DTYPE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _whole_scores(kind, d, lens, heads, group, seed, page=16):
    """Queries and keys of small whole numbers: their products are exact in fp32."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    table, pages = make_table(lens, page, seed)
    kc = torch.randint(-2, 3, (pages, page, heads, d[0]), generator=g).float().to(DTYPE[kind])
    vc = make_cache(pages, page, heads, d[1], kind, "token", seed + 1, device="cpu")
    q = torch.randint(-2, 3, (len(lens), heads * group, d[0]), generator=g).to(torch.bfloat16)
    return q.cuda(), kc.cuda(), vc.cuda(), table


def _largest_alone(q, kc, vc, table, lens, factor, v_unit):
    """O, its largest error in fp32 and LSE where only the keys of a row's largest score weigh
    anything: whole scores differ by at least one, times a factor of 2^20 or more."""
    heads, page = kc.shape[2], kc.shape[1]
    group = q.shape[1] // heads
    o = torch.zeros(*q.shape[:2], vc.shape[3], dtype=torch.float64, device=q.device)
    tol, lse = torch.zeros_like(o), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens):
        j = torch.arange(n, device=q.device)
        at = (table[b].long()[j // page], j % page)
        k = bits(kc)[at].view(kc.dtype).double()
        v = bits(vc)[at].view(vc.dtype).double() * v_unit
        for h in range(heads):
            rows = slice(h * group, (h + 1) * group)
            x = q[b, rows].double() @ k[:, h].T
            top = x.amax(-1, keepdim=True)
            w = (x == top).double()
            n_top = w.sum(-1, keepdim=True)
            o[b, rows] = w @ v[:, h] / n_top
            # weights of 1 and their count are exact; a sum of n_top products rounds at 2^-23 of
            # the sum of sizes n_top times (a tensor core truncates), and the factors of the
            # joins, the quotient and the product with it take a few roundings more
            tol[b, rows] = (n_top + 8) * 2.0 ** -23 * (w @ v[:, h].abs() / n_top)
            lse[b, rows] = (top * factor + torch.log(n_top))[:, 0]
    return o, tol, lse


@pytest.mark.parametrize("d", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("lens,heads,group", [([3, 70, 500, 3000], 2, 3), ([1, 900], 1, 16),
                                              ([20011], 1, 8)])
@pytest.mark.parametrize("kind,q_exp,k_exp,scale_exp", [
    ("bf16", 0, 0, 24), ("bf16", 0, 0, 40), ("bf16", 0, 0, 110), ("bf16", 50, 50, -60),
    ("e4m3", 0, 24, 0), ("e4m3", 0, 40, 0), ("e4m3", 0, 100, 0), ("e4m3", 0, 100, 10),
    ("e4m3", 100, 0, 0), ("e4m3", -20, 60, 0)])
def test_large_scores(ws, d, lens, heads, group, kind, q_exp, k_exp, scale_exp):
    """Scores of 2^24 to 2^119 times a whole number: the keys with the largest weigh all,
    evenly, whichever warps and parts they lie in."""
    q, kc, vc, table = _whole_scores(kind, d, lens, heads, group, seed=d[0] + heads)
    factor = 2.0 ** (q_exp + k_exp + scale_exp)
    unit = 1.0 if kind == "bf16" else 1 / 64
    scales = (None, None)
    keys = kc
    if kind == "e4m3":
        scales = (torch.full((heads,), 2.0 ** k_exp).cuda(), torch.full((heads,), unit).cuda())
    else:
        keys = kc * 2.0 ** k_exp
    cache = binding.PagedCache(keys, vc, *scales)
    o, lse = binding.decode(cache, q * 2.0 ** q_exp, table,
                            torch.tensor(lens, dtype=torch.int32).cuda(),
                            scale=2.0 ** scale_exp, workspace=ws)
    ro, tol, rl = _largest_alone(q, kc, vc, table, lens, factor, unit)
    assert torch.isfinite(lse).all() and torch.isfinite(o).all()
    assert ((o.double() - ro).abs() <= BF16_HALF * ro.abs() + tol * (1 + BF16_HALF)).all()
    # scale log2(e), times the score, times ln 2 (each factor and product rounded once, 2^-24)
    assert ((lse.double() - rl).abs() <= 6 * 2.0 ** -24 * rl.abs() + 2.0 ** -21).all()
    assert binding.attn_cache_status() == binding.ATTN_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 100, 9000])
def test_scores_beyond_fp32_make_the_row_not_finite(ws, kind, n):
    """A largest score above the largest fp32 value is no empty row; others stay as they are."""
    table, pages = make_table([n, 20], 16, 1)
    kc = torch.ones(pages, 16, 1, 64).to(DTYPE[kind]).cuda()
    vc = make_cache(pages, 16, 1, 64, kind, "token", 2)
    k_scale = torch.full((1,), 2.0 ** 100).cuda() if kind == "e4m3" else None
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16).cuda()
    q[1] = 0
    o, lse = binding.decode(binding.PagedCache(kc, vc, k_scale), q, table,
                            torch.tensor([n, 20], dtype=torch.int32).cuda(),
                            scale=2.0 ** (125 if kind == "bf16" else 25), workspace=ws)
    assert not torch.isfinite(lse[0]).any() and (lse[0] != -math.inf).all()
    assert not torch.isfinite(o[0]).any()
    assert torch.isfinite(o[1]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_an_infinite_query_of_an_empty_row(ws, kind):
    """A row that sees no key gives 0 and -inf, whatever its query holds."""
    table, pages = make_table([0, 20], 16, 1)
    kc, vc = (make_cache(pages, 16, 1, 64, kind, "token", s) for s in (1, 2))
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16).cuda() / 40
    q[0, 0], q[0, 1], q[0, 2, 3] = math.inf, math.nan, -math.inf
    o, lse = binding.decode(binding.PagedCache(kc, vc), q, table,
                            torch.tensor([0, 20], dtype=torch.int32).cuda(), workspace=ws)
    assert (o[0] == 0).all() and (lse[0] == -math.inf).all()
    assert torch.isfinite(o[1]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("d", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("octaves", [4, 12.3, 18.4, 22.4, 27])
@pytest.mark.parametrize("n,peak,heads", [(700, 0, 1), (700, 333, 2), (3000, 17, 1)])
def test_a_long_flat_tail_behind_one_large_weight(ws, d, kind, octaves, n, peak, heads):
    """One key weighs 2^octaves times each other and has a value of 0: what is left is the
    tail, and none of it may be lost beside the peak."""
    page, group = 16, 4
    table, pages = make_table([n], page, 3)
    g = torch.Generator(device="cpu").manual_seed(n + int(octaves))
    kc = torch.zeros(pages, page, heads, d[0])
    vc = torch.rand(pages, page, heads, d[1], generator=g) + 1
    at = (int(table[0, peak // page]), peak % page)
    kc[at[0], at[1], :, 0], vc[at[0], at[1]] = 256.0, 0.0
    kc, vc = kc.to(DTYPE[kind]).cuda(), vc.to(DTYPE[kind]).cuda()
    q = torch.zeros(1, heads * group, d[0], dtype=torch.bfloat16).cuda()
    q[..., 0] = 1.0
    scale = torch.tensor(octaves * math.log(2.0) / 256).item()
    o, lse = binding.decode(binding.PagedCache(kc, vc), q, table,
                            torch.tensor([n], dtype=torch.int32).cuda(), scale=scale, workspace=ws)
    ro, rl, _, _ = decode64(q, kc, vc, table, [n], page, scale)
    # a weight: rounded to 11 bits over an e4m3 cache, to 16 else; its exponent, up to 15 + octaves
    # in size, is a sum and a product in fp32, and the exponential is good to 2^-22; the sums
    # over n keys 2^-23 of the (positive) terms each at most
    rel = (2.0 ** -11 if kind == "e4m3" else 2.0 ** -16) + (15 + octaves) * 2.0 ** -23 \
        + 2.0 ** -22 + 2 * n * 2.0 ** -23
    assert ((o.double() - ro).abs() <= (BF16_HALF + rel * (1 + BF16_HALF)) * ro.abs()).all()
    assert ((lse.double() - rl).abs() <= rel + 2.0 ** -22 * rl.abs()).all()


@pytest.mark.parametrize("q_exp,k_exp,scale_exp,k_size", [(-122, 100, 28, -12), (124, -80, -64, 0),
                                                          (-122, 100, 20, -6), (60, 60, -125, 0)])
def test_e4m3_factors_of_which_two_alone_leave_the_range(ws, q_exp, k_exp, scale_exp, k_size):
    """The softmax scale, the keys' scale and the queries' size: their product is an ordinary
    factor, the product of two of them is not."""
    lens, page, heads, group, d = [1, 2, 20, 300], 16, 2, 4, 128
    table, pages = make_table(lens, page, 5)
    kc = (make_cache(pages, page, heads, d, "e4m3", "token", 6).float() * 2.0 ** k_size).to(
        torch.float8_e4m3fn)
    vc = make_cache(pages, page, heads, d, "e4m3", "token", 7)
    g = torch.Generator(device="cpu").manual_seed(8)
    q = (torch.randn(len(lens), heads * group, d, generator=g).clamp(-3, 3)
         * 2.0 ** q_exp).to(torch.bfloat16).cuda()
    ks, vs = torch.full((heads,), 2.0 ** k_exp).cuda(), torch.full((heads,), 1 / 64).cuda()
    scale = 2.0 ** scale_exp
    got = binding.decode(binding.PagedCache(kc, vc, ks, vs), q, table,
                         torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale, workspace=ws)
    check_decode(got, decode64(q, kc, vc, table, lens, page, scale, -1, ks, vs))
