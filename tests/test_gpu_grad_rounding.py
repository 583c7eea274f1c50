"""How often the gradients are rounded on their way: the norm of their error against fp64.

A rounding to bf16 of values spread evenly over their binades (in the logarithm) is off by
2^-8 / sqrt(3) * sqrt(3 / (8 ln 2)) = 1.66e-3 of their norm.  dQ and dK: dS is rounded once for its
products, and they are themselves: 2.35e-3 together.  dV and O: P, and they: as much.  D is the sum of
dO times an O that has been rounded, which in rows of few keys, as a causal problem has them, is up
to 0.9e-3 of dS: 2.52e-3.  One rounding more, of P or of dP - D before their product, makes that 2.9e-3
and above, two of them 3.3e-3."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding

pytestmark = pytest.mark.gpu

BOUND = {False: 2.5e-3, True: 2.7e-3}  # by causal


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()


def gradients64(q, k, v, dO, causal):
    group = q.shape[2] // k.shape[2]
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    heads = lambda t, g: t.transpose(1, 2).repeat_interleave(g, 1)
    x = heads(leaves[0], 1) @ heads(leaves[1], group).mT / math.sqrt(q.shape[-1])
    if causal:
        x = x.masked_fill(torch.ones(x.shape[-2:], dtype=torch.bool, device=x.device).triu(1), -math.inf)
    o = (torch.softmax(x, -1) @ heads(leaves[2], group)).transpose(1, 2)
    o.backward(dO.double())
    return [o.detach()] + [t.grad for t in leaves]


def error(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("det", [False, True])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (6, 1)])
@pytest.mark.parametrize("d", [(64, 64), (128, 128), (192, 128)])
def test_one_rounding_each(d, heads, det, causal):
    g = torch.Generator(device="cuda").manual_seed(d[0] + heads[0])
    rand = lambda h, w: torch.randn(2, 512, h, w, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v, dO = rand(heads[0], d[0]), rand(heads[1], d[0]), rand(heads[1], d[1]), rand(heads[0], d[1])
    o, lse = binding.forward(q, k, v, causal=causal)
    got = (o,) + tuple(binding.backward(q, k, v, o, dO, lse, causal=causal, deterministic=det))
    for name, a, b in zip(("O", "dQ", "dK", "dV"), got, gradients64(q, k, v, dO, causal)):
        assert error(a, b) <= BOUND[causal], name


@pytest.mark.parametrize("causal", [False, True])
def test_one_rounding_each_pair_of_ctas(causal):
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, dO = (torch.randn(1, 640, 4, 128, generator=g, device="cuda").to(torch.bfloat16)
                   for _ in range(4))
    o, lse = binding.forward(q, k, v, causal=causal)
    binding.attn_debug_set_bwd_variant(binding.BWD_CTA_PAIR)
    try:
        got = binding.backward(q, k, v, o, dO, lse, causal=causal)
        torch.cuda.synchronize()
    finally:
        binding.attn_debug_set_bwd_variant(binding.BWD_AUTO)
    for name, a, b in zip(("dQ", "dK", "dV"), got, gradients64(q, k, v, dO, causal)[1:]):
        assert error(a, b) <= BOUND[causal], name
