"""Sequences of a batch that hold infinities or NaN: in the forward the others, some of whose tiles share
rows with theirs, keep every bit of what they are without."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()


CASES = [
    # lengths of queries, of keys (None: the same), fixed, hq, hk, (dqk, dv), causal, window
    ([77, 1, 300, 0, 129, 200, 128, 5], None, False, 4, 4, (64, 64), True, None),
    ([77, 1, 300, 0, 129, 200, 128, 5], None, False, 8, 2, (128, 128), True, None),
    ([200, 33, 400, 1, 256], None, False, 6, 1, (192, 128), False, None),
    ([90, 5, 64, 130], [300, 5, 129, 140], False, 4, 2, (128, 128), True, None),
    ([90, 0, 64, 130], [300, 70, 129, 140], False, 4, 4, (64, 64), False, None),
    ([500, 150, 270], None, False, 4, 2, (128, 128), False, (60, 20)),
    ([500, 150, 270], None, False, 3, 3, (192, 128), True, (100, 0)),
    ([130] * 4, None, True, 4, 4, (128, 128), True, None),
    ([77] * 3, None, True, 8, 2, (64, 64), False, None),
    ([40] * 3, [200] * 3, True, 3, 3, (192, 128), True, None),
    ([5, 33, 9, 64, 1] * 60, None, False, 4, 2, (64, 64), True, None),  # several items to a CTA
    ([700, 1100, 33] * 8, None, False, 8, 2, (128, 128), False, None),
]


def _inputs(case):
    lens, lens_k, fixed, hq, hk, (dqk, dv), _, _ = CASES[case]
    lens_k = lens if lens_k is None else lens_k
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda rows, h, d: torch.randn(rows, h, d, generator=g, device="cuda").to(torch.bfloat16)
    return {"q": rand(sum(lens), hq, dqk), "k": rand(sum(lens_k), hk, dqk),
            "v": rand(sum(lens_k), hk, dv)}, lens, lens_k


def _offsets(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def _forward(case, t, block_mask=None):
    """O and LSE (T, H) over flat rows."""
    lens, lens_k, fixed, hq, hk, d, causal, window = CASES[case]
    kw = dict(causal=causal, window=window)
    if fixed:
        t = {n: x.unflatten(0, (len(lens), -1)) for n, x in t.items()}
    else:
        kw["cu_seqlens"] = _offsets(lens)
        if lens_k is not None:
            kw["cu_seqlens_k"] = _offsets(lens_k)
    if block_mask is not None:
        kw["block_mask"] = block_mask
    o, lse = binding.forward(t["q"], t["k"], t["v"], **kw)
    assert binding.attn_fwd_status() == binding.ATTN_OK
    return (o.flatten(0, 1), lse.transpose(1, 2).flatten(0, 1)) if fixed else (o, lse.t())


def _poisoned(t, lens, lens_k, b, names, value):
    bad = {n: x.clone() for n, x in t.items()}
    for n in names:
        c = _offsets(lens if n == "q" else lens_k)
        bad[n][c[b]:c[b + 1]] = value
    return bad


@pytest.mark.parametrize("case", range(len(CASES)))
def test_others_keep_their_bits(case):
    t, lens, lens_k = _inputs(case)
    clean = _forward(case, t)
    assert all(torch.isfinite(x).all() for x in clean)
    cu = _offsets(lens)
    for b in range(min(len(lens), 12)):
        for names, value in (("qkv", NAN), ("v", INF), ("k", -INF), ("q", INF)):
            got = _forward(case, _poisoned(t, lens, lens_k, b, names, value))
            keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
            keep[cu[b]:cu[b + 1]] = False
            for x, y in zip(clean, got):
                assert torch.equal(x[keep], y[keep]), (b, names, value)


def test_others_keep_their_bits_under_a_block_mask():
    """Tiles that the mask drops, the shared ones of some sequences and heads among them."""
    t, lens, lens_k = _inputs(0)
    blocks = -(-max(lens) // binding.BLOCK)
    g = torch.Generator().manual_seed(1)
    mask = (torch.rand(len(lens), 4, blocks, blocks, generator=g) < 0.6).to(torch.uint8)
    mask[:, 0] = torch.eye(blocks, dtype=torch.uint8)
    mask = mask.cuda()
    clean = _forward(0, t, mask)
    cu = _offsets(lens)
    for b in range(len(lens)):
        got = _forward(0, _poisoned(t, lens, lens_k, b, "qkv", NAN), mask)
        keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
        keep[cu[b]:cu[b + 1]] = False
        for x, y in zip(clean, got):
            assert torch.equal(x[keep], y[keep]), b
