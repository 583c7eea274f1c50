"""Prefill where tiles that come by rows lie between tiles that come by boxes: pages outside the
cache in tiles that every row sees, several to a CTA's share of the work."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import bits
from tests.test_gpu_prefill import check, prefill64, setup

pytestmark = pytest.mark.gpu

TILE = 128
# Key tiles of a sequence with one page outside the cache each.
PATTERNS = [(), (0, 2), (0, 4), (), (1, 3, 5), (0, 1, 2, 3), (2, 7), ()]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()


def without(kc, vc, table, length, page, gone):
    """The sequence's keys but those of pages `gone`, in caches of one page each."""
    j = torch.tensor([i for i in range(length) if i // page not in gone]).cuda()
    at = (table.long()[j // page], j % page)
    out = []
    for c in (kc, vc):
        one = torch.zeros((1, len(j)) + c.shape[2:], dtype=c.dtype, device="cuda")
        bits(one)[0] = bits(c)[at]
        out.append(one)
    return out, len(j)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [(128, 128), (64, 64), (192, 128)])
@pytest.mark.parametrize("page,new", [(16, 40), (64, 5)])
def test_bad_pages_between_whole_tiles(kind, d, page, new):
    """24 sequences and 8 key heads make 192 units of 13 or more tiles, so a share has 15 of them
    and more.  Sequences whose pages are all there have the bits of a call without bad pages; the
    others are attended without the keys of theirs."""
    heads, group, B = 8, 4, 24
    lens = [1500 + 37 * (b % 5) for b in range(B)]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(7, heads, group, *d, page, kind, "token",
                                                    [new] * B, lens, poison=False)
    good = binding.prefill(cache, q, table, lens_d)
    assert binding.attn_cache_status() == binding.ATTN_OK
    gone = [[(t * TILE + (17 * b + 31 * t) % TILE) // page for t in PATTERNS[b % 8]]
            for b in range(B)]
    host = table.cpu()
    for b in range(B):
        for i, p in enumerate(gone[b]):
            host[b, p] = (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31)[i % 4]
    broken = host.cuda()
    o, lse = binding.prefill(cache, q, broken, lens_d)
    assert binding.attn_cache_status() == binding.ATTN_ERR_BAD_PAGE
    again = binding.prefill(cache, q, broken, lens_d)
    assert binding.attn_cache_status() == binding.ATTN_ERR_BAD_PAGE
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    scale = 1.0 / math.sqrt(d[0])
    for b in range(B):
        rows = slice(b * new, (b + 1) * new)
        if not gone[b]:
            assert torch.equal(o[rows], good[0][rows]) and torch.equal(lse[rows], good[1][rows])
            continue
        (k1, v1), n = without(kc, vc, table[b], lens[b], page, gone[b])
        ref = prefill64(q[rows], k1, v1, torch.zeros(1, 1, dtype=torch.int32).cuda(), [n], [new], n,
                        scale, -1, ks, vs)
        check((o[rows], lse[rows]), ref, f"sequence {b}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("length", [-5, 0])
def test_neighbours_of_an_empty_sequence(kind, length):
    """A length of 0 or below changes where the work is cut: the other sequences keep the bounds."""
    heads, group, page, d = 2, 2, 16, 64
    new, lens = [5, 5, 5], [100, 100, 300]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(4, heads, group, d, d, page, kind, "token", new,
                                                    lens, poison=False)
    lens_d[0] = length
    got = binding.prefill(cache, q, table, lens_d)
    assert binding.attn_cache_status() == binding.ATTN_OK
    check(got, prefill64(q, kc, vc, table, [length] + lens[1:], new, page, 0.125, -1, ks, vs))
