"""Prefill over batches whose units have one query tile and two in every order (over an e4m3 cache the
second tile's place serves the cache's rows while units have one)."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.test_gpu_prefill import check, prefill64, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("d", [(128, 128), (192, 128), (64, 64)])
@pytest.mark.parametrize("order", [0, 1, 2])
def test_single_tiles_and_pairs_in_turn(kind, d, order):
    """With groups of four a tile has 32 tokens: 33 and more are a unit of two.  120 sequences and 8
    key heads are 960 units and more, six to a CTA; one key tile each, or several."""
    heads, group, page = 8, 4, 16
    runs = [[1, 40], [1, 5, 64], [1, 2, 3, 33, 50, 1, 70]][order]
    new = (runs * 120)[:120]
    lens = [n + (i * 37) % (90 if i % 3 else 500) for i, n in enumerate(new)]
    cache, q, kc, vc, ks, vs, table, lens_d = setup(order, heads, group, *d, page, kind, "token", new,
                                                    lens)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    got = binding.prefill(cache, q, table, lens_d, cu_seqlens=cu)
    assert binding.attn_cache_status() == binding.ATTN_OK
    check(got, prefill64(q, kc, vc, table, lens, new, page, 1.0 / math.sqrt(d[0]), -1, ks, vs))
    again = binding.prefill(cache, q, table, lens_d, cu_seqlens=cu)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
