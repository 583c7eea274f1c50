"""Prefill over a paged cache against 64-bit references.  Slots that no row sees hold NaN."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import (BF16_HALF, bits, make_cache, make_table, nan_bits,
                                poison_unseen)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()


def prefill64(q, kc, vc, table, lens, new, page, scale, window=-1, ks=None, vs=None):
    """O, LSE and bounds of their errors, sequence by sequence in fp64.  The bounds:
      scores: fp32 sums of d products, each rounding at 2^-23 of the sum of absolute values, and
        the rounding of s x (2^-22 of it, scale and exponent);
      weights: bf16, 2^-8 of each at most; the exponential itself 2^-22;
      the sum over n keys: n 2^-23; O: one rounding to bf16."""
    T, Hq, dqk = q.shape
    heads, dv = kc.shape[2], vc.shape[3]
    G = Hq // heads
    o = torch.zeros(T, Hq, dv, dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
    a = 0
    for b, (n, m) in enumerate(zip(new, lens)):
        rows = slice(a, a + n)
        a += n
        if m <= 0 or n == 0:
            continue
        j = torch.arange(m, device=q.device)
        at = (table[b].long()[j // page], j % page)
        pos = torch.arange(m - n, m, device=q.device)[:, None]
        seen = j <= pos
        if window >= 0:
            seen &= j >= pos - window
        k = bits(kc)[at].view(kc.dtype).double()
        v = bits(vc)[at].view(vc.dtype).double()
        if ks is not None:
            k = k * ks.double()[:, None]
        if vs is not None:
            v = v * vs.double()[:, None]
        used = seen.any(0)[:, None, None]
        k, v = torch.where(used, k, 0.0), torch.where(used, v, 0.0)
        qb = q[rows].double().view(n, heads, G, dqk).permute(1, 2, 0, 3)  # heads, G, n, d
        k, v = k.permute(1, 2, 0)[:, None], v.permute(1, 0, 2)[:, None]
        x = (qb @ k * scale).masked_fill(~seen, -math.inf)
        mag = (qb.abs() @ k.abs() * scale).masked_fill(~seen, 0.0).amax(-1)
        top = x.masked_fill(~seen, 0.0).abs().amax(-1)
        lb = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(lb == -math.inf, 0.0, lb)[..., None])
        ob, ab = p @ v, p @ v.abs()
        dx = (dqk + 2) * 2.0 ** -23 * mag + 2.0 ** -22 * top
        rel = 2.0 ** -22 + 2 * dx + m * 2.0 ** -23
        tol = ab * (rel + BF16_HALF)[..., None]
        back = lambda t: t.permute(2, 0, 1, *range(3, t.dim())).reshape(n, Hq, *t.shape[3:])
        o[rows], lse[rows] = back(ob), back(lb)
        tol_o[rows] = back(BF16_HALF * ob.abs() + tol * (1 + BF16_HALF))
        tol_l[rows] = back(rel + 2.0 ** -22 * torch.where(lb == -math.inf, 0.0, lb).abs())
    return o, lse, tol_o, tol_l


def check(got, ref, where=""):
    o, lse = got
    ro, rl, to, tl = ref
    empty = rl == -math.inf
    assert torch.isfinite(o).all(), where
    if lse is not None:
        assert torch.equal(lse.double() == -math.inf, empty), where
        over = ((lse.double() - rl).abs() - tl)[~empty]
        assert over.numel() == 0 or (over <= 0).all(), f"{where}: LSE over by {over.max()}"
    over = (o.double() - ro).abs() - to
    assert (over <= 0).all(), f"{where}: O over by {over.max()} at {over.argmax()}"


def setup(seed, heads, group, dqk, dv, page, kind, order, new, lens, window=-1, poison=True):
    g = torch.Generator(device="cpu").manual_seed(seed)
    table, pages = make_table([max(0, m) for m in lens], page, seed + 1)
    kc = make_cache(pages, page, heads, dqk, kind, order, seed + 2)
    vc = make_cache(pages, page, heads, dv, kind, order, seed + 3)
    ks = vs = None
    if kind == "e4m3":
        ks = ((1 + torch.rand(heads, generator=g)) / 48).cuda()
        vs = ((1 + torch.rand(heads, generator=g)) / 48).cuda()
    if poison:
        keep = torch.zeros(kc.shape[:2], dtype=torch.bool)
        for b, (n, m) in enumerate(zip(new, lens)):
            for j in range(max(0, m - n - window) if window >= 0 else 0, m):
                keep[int(table[b, j // page]), j % page] = True
        for c in (kc, vc):
            bits(c)[~keep.cuda()] = nan_bits(c)
    q = torch.randn(sum(new), heads * group, dqk, generator=g).to(torch.bfloat16).cuda()
    cache = binding.PagedCache(kc, vc, ks, vs)
    return cache, q, kc, vc, ks, vs, table, torch.tensor(lens, dtype=torch.int32).cuda()


CASES = [
    # heads, group, (dqk, dv), page, new, lens, window
    (1, 1, (128, 128), 16, [1], [1], -1),
    (2, 4, (128, 128), 64, [5, 5, 5], [5, 130, 1000], -1),
    (2, 4, (64, 64), 16, [77, 1, 0, 300], [77, 400, 50, 300], -1),
    (1, 3, (128, 128), 24, [43, 200], [600, 200], 100),
    (3, 5, (64, 64), 1, [30, 2], [150, 2], -1),
    (2, 7, (192, 128), 32, [40, 19, 1], [41, 300, 900], -1),
    (4, 1, (128, 128), 128, [129, 257], [129, 700], 0),
    (2, 12, (128, 128), 256, [11, 64], [2000, 64], 127),
    (1, 16, (192, 128), 8, [100], [1200], -1),
    (1, 128, (128, 128), 64, [3, 1], [100, 700], -1),
    (1, 100, (64, 64), 12, [2, 5], [33, 260], 40),
    (8, 4, (128, 128), 64, [1] * 9, [1, 0, 64, 65, 127, 128, 129, 3000, 17], -1),
    (2, 2, (128, 128), 16, [6, 300, 4], [0, 250, 2], -1),   # fewer keys than new tokens
]


@pytest.mark.parametrize("kind,order", [("bf16", "token"), ("bf16", "head"), ("bf16", "joint"),
                                        ("e4m3", "token"), ("e4m3", "head")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_prefill(case, kind, order):
    heads, group, (dqk, dv), page, new, lens, window = CASES[case]
    if order == "joint" and dqk != dv:
        pytest.skip("one buffer for both sides")
    cache, q, kc, vc, ks, vs, table, lens_d = setup(case, heads, group, dqk, dv, page, kind, order,
                                                    new, lens, window)
    scale = 1.0 / math.sqrt(dqk)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    ws = binding.prefill_workspace()
    got = binding.prefill(cache, q, table, lens_d, window_left=window, cu_seqlens=cu, workspace=ws)
    assert binding.attn_cache_status() == binding.ATTN_OK
    ref = prefill64(q, kc, vc, table, lens, new, page, scale, window, ks, vs)
    check(got, ref)
    again = binding.prefill(cache, q, table, lens_d, window_left=window, cu_seqlens=cu,
                            workspace=ws)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    if len(set(new)) == 1:  # the same without offsets
        even = binding.prefill(cache, q, table, lens_d, window_left=window, workspace=ws)
        assert torch.equal(got[0], even[0]) and torch.equal(got[1], even[1])
