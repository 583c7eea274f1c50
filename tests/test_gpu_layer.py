"""The operators together, as a layer uses them: in training, norms with the rotation, grouped
attention and the gradients of both; in serving, prompts normed and appended in chunks, attended by
prefill, then generated from token by token."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import (BF16_HALF, check_decode, decode64, inv_freq, make_cache, make_table,
                                rotate64)
from tests.test_gpu_prefill import check, prefill64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()
    binding.attn_fwd_status()


def _rand(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("packed", [False, True])
def test_training_layer(packed):
    """norm_rope -> forward -> backward -> norm_rope_backward over the slices of one projection, and
    every gradient against autograd through the same formulas in fp64."""
    lens, hq, hk, d = [150, 1, 77], 6, 2, 128
    T = sum(lens)
    cu = [sum(lens[:i]) for i in range(4)]
    g = torch.Generator().manual_seed(0)
    row = _rand(g, T, (hq + 2 * hk) * d)
    q, k, v = (t.unflatten(1, (-1, d)) for t in row.split([hq * d, hk * d, hk * d], 1))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    dO = _rand(g, T, hq, d)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    freq = inv_freq(d)
    norm, rot = binding.HeadNorm(wq, wk, eps=1e-6), binding.Rotation(freq)
    qn, kn = binding.norm_rope(q, k, norm, rot, cu_seqlens=cu)
    o, lse = binding.forward(qn, kn, v, causal=True, cu_seqlens=cu)
    dqn, dkn, dv = binding.backward(qn, kn, v, o, dO, lse, causal=True, cu_seqlens=cu)
    dq, dk, dwq, dwk = binding.norm_rope_backward(q, k, dqn, dkn, norm, rot, cu_seqlens=cu)
    assert binding.attn_fwd_status() == binding.ATTN_OK

    leaves = [t.double().requires_grad_() for t in (q, k, v, wq, wk)]
    unit = lambda x, w: w * x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    turned = [rotate64(unit(x, w), pos, freq, 0, False)[0]
              for x, w in ((leaves[0], leaves[3]), (leaves[1], leaves[4]))]
    outs = []
    for b in range(3):
        r = slice(cu[b], cu[b + 1])
        wide = lambda t: t[r].repeat_interleave(hq // hk, 1).transpose(0, 1)
        s = turned[0][r].transpose(0, 1) @ wide(turned[1]).transpose(1, 2) / math.sqrt(d)
        n = lens[b]
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).cuda().triu(1), -math.inf)
        outs.append((torch.softmax(s, -1) @ wide(leaves[2])).transpose(0, 1))
    torch.cat(outs).backward(dO.double())
    assert (o.double() - torch.cat(outs)).norm() / torch.cat(outs).norm() <= 5e-3 + 2 * BF16_HALF
    # the backward's own tolerance (1e-2 of the norm), and the roundings of the turned q, k and of the
    # gradients on the way (2^-8 each at most)
    for got, leaf in zip((dq, dk, dv, dwq, dwk), leaves):
        assert (got.double() - leaf.grad).norm() / leaf.grad.norm() <= 1e-2 + 3 * BF16_HALF


@pytest.mark.parametrize("d,begin,dim,inter", [((64, 64), 0, 64, False),
                                               ((128, 128), 0, 128, False),
                                               ((192, 128), 128, 64, True)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("normed", [False, True])
def test_chunks_then_generate(d, begin, dim, inter, kind, normed):
    dqk, dv = d
    heads, Hq, page = 2, 8, 16
    chunks = [[30, 100, 1], [40, 7, 0], [0, 60, 5]]  # new tokens of three sequences, step by step
    total = [sum(c[b] for c in chunks) + 2 for b in range(3)]
    g = torch.Generator().manual_seed(dqk)
    table, pages = make_table(total, page, 3)
    kc = make_cache(pages, page, heads, dqk, kind, "token", 4)
    vc = make_cache(pages, page, heads, dv, kind, "token", 5)
    unit = torch.full((heads,), 1 / 64).cuda() if kind == "e4m3" else None
    cache = binding.PagedCache(kc, vc, unit, unit)
    rot = binding.Rotation(inv_freq(dim), begin=begin, interleaved=inter)
    wq, wk = ((1 + 0.2 * torch.randn(dqk, generator=g)).cuda() for _ in range(2))
    norm = binding.HeadNorm(wq, wk) if normed else None
    ws, dws = binding.prefill_workspace(), binding.decode_workspace()
    scale = 1 / math.sqrt(dqk)
    have = [0, 0, 0]
    rows = {b: [] for b in range(3)}  # queries, keys, values as projected, and O
    for new in chunks:
        T = sum(new)
        cu = [sum(new[:i]) for i in range(4)]
        have = [a + n for a, n in zip(have, new)]
        lens = torch.tensor(have, dtype=torch.int32).cuda()
        q, k, v = _rand(g, T, Hq, dqk), _rand(g, T, heads, dqk), _rand(g, T, heads, dv)
        qt = binding.cache_append(cache, k, v, table, lens, q=q, rotation=rot, cu_seqlens=cu,
                                  norm=norm)
        got = binding.prefill(cache, qt, table, lens, cu_seqlens=cu, workspace=ws)
        check(got, prefill64(qt, kc, vc, table, have, new, page, scale, -1, unit, unit))
        for b in range(3):
            r = slice(cu[b], cu[b + 1])
            rows[b].append((q[r], k[r], v[r], got[0][r], got[1][r]))
    if kind == "bf16":  # (an 8-bit cache holds other keys than the forward sees)
        full = [torch.cat([torch.cat([c[i] for c in rows[b]]) for b in range(3)]) for i in range(5)]
        cu = [sum(have[:i]) for i in range(4)]
        if normed:
            qr, kr = binding.norm_rope(full[0], full[1], norm, rot, cu_seqlens=cu)
        else:
            qr, kr = binding.rope(full[0], full[1], rot, cu_seqlens=cu)
        o, lse = binding.forward(qr, kr, full[2], causal=True, cu_seqlens=cu)
        # both round their weights and O to bf16 once each
        top = full[2].double().abs().amax()
        assert ((o.double() - full[3].double()).abs() <= BF16_HALF * (2 * o.double().abs() + 4 * top)).all()
        assert (o.double() - full[3].double()).norm() / o.double().norm() <= 5e-3
        assert (lse.t() - full[4]).abs().max() <= 1e-4
    # a token each, by decode and by prefill
    for _ in range(2):
        have = [n + 1 for n in have]
        lens = torch.tensor(have, dtype=torch.int32).cuda()
        q, k, v = _rand(g, 3, Hq, dqk), _rand(g, 3, heads, dqk), _rand(g, 3, heads, dv)
        qt = binding.cache_append(cache, k, v, table, lens, q=q, rotation=rot, norm=norm)
        check_decode(binding.decode(cache, qt, table, lens, workspace=dws),
                     decode64(qt, kc, vc, table, have, page, scale, -1, unit, unit))
        check(binding.prefill(cache, qt, table, lens, workspace=ws),
              prefill64(qt, kc, vc, table, have, [1, 1, 1], page, scale, -1, unit, unit))
    assert binding.attn_cache_status() == binding.ATTN_OK


def test_two_calls_at_once():
    """Calls on two streams, each with its workspace, and two captured graphs replayed side by side."""
    heads, Hq, d, page = 4, 16, 128, 32
    lens = [3000, 777]
    table, pages = make_table(lens, page, 3)
    kc = make_cache(pages, page, heads, d, "bf16", "token", 4)
    vc = make_cache(pages, page, heads, d, "bf16", "token", 5)
    cache = binding.PagedCache(kc, vc)
    lens_d = torch.tensor(lens, dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(1)
    qs = [_rand(g, 2 * n, Hq, d) for n in (40, 3)]
    x = [_rand(g, 1, 500, h, d) for h in (Hq, heads, heads)]
    want = [binding.prefill(cache, q, table, lens_d) for q in qs]
    full = binding.forward(*x, causal=True)
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws = [binding.prefill_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for i in range(2):
            outs.append((i, binding.prefill(cache, qs[i], table, lens_d, workspace=ws[i],
                                            stream=streams[i])))
        outs.append((2, binding.forward(*x, causal=True, stream=streams[2])))
    torch.cuda.synchronize()
    graphs, kept = [], []
    for i in range(3):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for _ in range(3):
                kept.append((i, binding.prefill(cache, qs[i], table, lens_d, workspace=ws[i])
                             if i < 2 else binding.forward(*x, causal=True)))
        graphs.append(gr)
    for _ in range(3):
        for i, gr in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                gr.replay()
    torch.cuda.synchronize()
    for i, (o, lse) in outs + kept:
        a, b = want[i] if i < 2 else full
        assert torch.equal(o, a) and torch.equal(lse, b)
    assert binding.attn_cache_status() == binding.ATTN_OK
    assert binding.attn_fwd_status() == binding.ATTN_OK
