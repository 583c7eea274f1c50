"""The operators together, as a program that serves a model uses them: prompts rotated and
attended by the forward, appended to a paged cache, then tokens generated one by one (append
with the rotation on the way, then decode), eagerly and as one captured step."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import (BF16_HALF, check_decode, decode64, inv_freq, make_cache,
                                make_table)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()


def _rand(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("d,begin,dim,inter", [((64, 64), 0, 64, False),
                                               ((128, 128), 0, 128, False),
                                               ((192, 128), 128, 64, True)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,group", [(4, 1), (2, 4)])
def test_prefill_then_generate(d, begin, dim, inter, kind, heads, group):
    dqk, dv = d
    page, steps = 16, 4
    prompts = [37, 1, 16, 200]
    B, Hq = len(prompts), heads * group
    g = torch.Generator(device="cpu").manual_seed(dqk + heads)
    final = [n + steps for n in prompts]
    table, pages = make_table(final, page, 3)
    kc = make_cache(pages, page, heads, dqk, kind, "token", 4)
    vc = make_cache(pages, page, heads, dv, kind, "token", 5)
    unit = torch.full((heads,), 1 / 64).cuda() if kind == "e4m3" else None
    cache = binding.PagedCache(kc, vc, unit, unit)
    rot = binding.Rotation(inv_freq(dim), begin=begin, interleaved=inter)
    ws = binding.decode_workspace()
    cu = [sum(prompts[:i]) for i in range(B + 1)]
    T = cu[-1]
    scale = 1.0 / math.sqrt(dqk)

    # prompts
    q, k, v = _rand(g, T, Hq, dqk), _rand(g, T, heads, dqk), _rand(g, T, heads, dv)
    lens = torch.tensor(prompts, dtype=torch.int32).cuda()
    q_rot = binding.cache_append(cache, k, v, table, lens, q=q, rotation=rot, cu_seqlens=cu)
    q2, k_rot = binding.rope(q, k, rot, cu_seqlens=cu)
    assert torch.equal(q_rot, q2)  # one arithmetic in both
    wide = lambda t: t.repeat_interleave(group, 1).contiguous()
    o, lse = binding.forward(q_rot, wide(k_rot), wide(v), causal=True, cu_seqlens=cu)
    # the forward's last row of each prompt is what a decode over the cache gives
    last = torch.tensor([c - 1 for c in cu[1:]]).cuda()
    od, ld = binding.decode(cache, q_rot[last].contiguous(), table, lens, workspace=ws)
    ref = decode64(q_rot[last], kc, vc, table, prompts, page, scale, -1, unit, unit)
    check_decode((od, ld), ref)
    if kind == "bf16":  # (an 8-bit cache holds other keys than the forward saw)
        for b in range(B):
            rows = torch.arange(cu[b], cu[b + 1]).cuda()
            at = (table[b].long()[torch.arange(prompts[b]).cuda() // page],
                  torch.arange(prompts[b]).cuda() % page)
            assert torch.equal(kc[at], k_rot[rows]) and torch.equal(vc[at], v[rows])
        # both within their bounds of the exact value: the forward rounds its probabilities
        # and O to bf16 once each (of at most the sum of |p v|, here at most max |v|)
        off = (o[last].double() - ref[0]).abs()
        top = wide(v).double().abs().amax()
        assert (off <= BF16_HALF * (ref[0].abs() + 2 * top)).all()
        assert (lse.t()[last].double() - ref[1]).abs().max() <= 1e-4

    # generation
    have = list(prompts)
    outs = []
    for _ in range(steps):
        row = _rand(g, B, Hq * dqk + heads * (dqk + dv))
        qs, ks, vs = row.split([Hq * dqk, heads * dqk, heads * dv], 1)
        lens += 1
        have = [n + 1 for n in have]
        qs = binding.cache_append(cache, ks.unflatten(1, (heads, dqk)),
                                  vs.unflatten(1, (heads, dv)), table, lens,
                                  q=qs.unflatten(1, (Hq, dqk)), rotation=rot)
        got = binding.decode(cache, qs, table, lens, workspace=ws)
        check_decode(got, decode64(qs, kc, vc, table, have, page, scale, -1, unit, unit))
        outs.append((row, got))
    assert binding.attn_cache_status() == binding.ATTN_OK

    # the same steps again as one captured step, from the prompts on
    lens.copy_(torch.tensor(prompts, dtype=torch.int32))
    row = outs[0][0].clone()
    qs, ks, vs = row.split([Hq * dqk, heads * dqk, heads * dv], 1)
    q_out = torch.empty(B, Hq, dqk, dtype=torch.bfloat16, device="cuda")
    dst = (torch.empty(B, Hq, dv, dtype=torch.bfloat16, device="cuda"),
           torch.empty(B, Hq, device="cuda"))

    def step():
        lens.add_(1)
        binding.cache_append(cache, ks.unflatten(1, (heads, dqk)), vs.unflatten(1, (heads, dv)),
                             table, lens, q=qs.unflatten(1, (Hq, dqk)), rotation=rot, q_out=q_out)
        binding.decode(cache, q_out, table, lens, workspace=ws, out=dst)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for src, want in outs:
        row.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dst[0], want[0]) and torch.equal(dst[1], want[1])
    assert binding.attn_cache_status() == binding.ATTN_OK


def test_training_step_with_rotation():
    """rope -> forward -> backward -> inverse rope: the gradients of the unrotated queries and
    keys, against autograd through the same formulas in fp64."""
    B, T, H, D = 1, 96, 2, 64
    g = torch.Generator(device="cpu").manual_seed(0)
    q, k, v, dO = (_rand(g, B, T, H, D) for _ in range(4))
    freq = inv_freq(D)
    rot = binding.Rotation(freq)
    qr, kr = binding.rope(q, k, rot)
    o, lse = binding.forward(qr, kr, v, causal=True)
    dqr, dkr, dv = binding.backward(qr, kr, v, o, dO, lse, causal=True)
    dq, dk = binding.rope(dqr, dkr, rot, inverse=True)
    assert binding.attn_fwd_status() == binding.ATTN_OK

    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    ang = torch.arange(T).double().cuda()[:, None] * torch.tensor(freq).double().cuda()
    cos, sin = torch.cos(ang)[None, :, None], torch.sin(ang)[None, :, None]

    def turn(x):
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)

    s = torch.einsum("bthd,bshd->bhts", turn(leaves[0]), turn(leaves[1])) / math.sqrt(D)
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool).cuda().triu(1), -math.inf)
    ref = torch.einsum("bhts,bshd->bthd", torch.softmax(s, -1), leaves[2])
    ref.backward(dO.double())
    # the backward's own tolerance (1e-2 of the norm), and the roundings of the rotated q, k and
    # of the gradients on the way (2^-8 each at most)
    for got, leaf in zip((dq, dk, dv), leaves):
        err = (got.double() - leaf.grad).norm() / leaf.grad.norm()
        assert err <= 1e-2 + 3 * BF16_HALF
