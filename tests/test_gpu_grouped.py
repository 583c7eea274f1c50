"""Grouped heads: the forward and backward against the formulas in fp64 (a padded-free loop over
sequences and key heads, gradients by autograd), and against the same call on repeated keys."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.gpu_common import TOL_GRAD, TOL_LSE, TOL_O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()


def _inputs(seed, lens, hq, hk, dqk, dv, packed, fixed, lens_k=None):
    g = torch.Generator(device="cpu").manual_seed(seed)
    lens_k = lens if lens_k is None else lens_k
    rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    rows = (len(lens), lens[0]) if fixed else (sum(lens),)
    rows_k = (len(lens), lens_k[0]) if fixed else (sum(lens_k),)
    if packed:
        x = rand(*rows, hq * dqk + hk * (dqk + dv))
        q, k, v = x.split([hq * dqk, hk * dqk, hk * dv], -1)
        q, k, v = (t.unflatten(-1, (h, -1)) for t, h in ((q, hq), (k, hk), (v, hk)))
    else:
        q, k, v = rand(*rows, hq, dqk), rand(*rows_k, hk, dqk), rand(*rows_k, hk, dv)
    return q, k, v, rand(*rows, hq, dv)


def _reference(q, k, v, dO, lens, lens_k, scale, causal, window):
    """O, LSE (Hq, T) and gradients in fp64, over flat rows."""
    flat = lambda x: x.reshape(-1, *x.shape[-2:]).double()
    q, k, v = (flat(t).requires_grad_() for t in (q, k, v))
    group = q.shape[1] // k.shape[1]
    outs, stats = [], []
    a = b = 0
    for n, m in zip(lens, lens_k):
        qs, ks, vs = q[a:a + n], k[b:b + m], v[b:b + m]
        i = torch.arange(n, device="cuda")[:, None] + (m - n)
        j = torch.arange(m, device="cuda")
        seen = torch.ones(n, m, dtype=torch.bool, device="cuda")
        wl, wr = (-1, -1) if window is None else window
        if causal:
            seen &= j <= i
        if wl >= 0:
            seen &= j >= i - wl
        if wr >= 0:
            seen &= j <= i + wr
        wide = lambda t: t.repeat_interleave(group, 1).transpose(0, 1)
        x = (qs.transpose(0, 1) @ wide(ks).transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
        outs.append((torch.softmax(x, -1) @ wide(vs)).transpose(0, 1))
        stats.append(torch.logsumexp(x, -1))
        a, b = a + n, b + m
    o, lse = torch.cat(outs), torch.cat(stats, 1)
    o.backward(flat(dO))
    return o.detach(), lse.detach(), q.grad, k.grad, v.grad


def _norm_err(got, ref):
    got = got.reshape(ref.shape).double()
    return float((got - ref).norm() / ref.norm().clamp(min=1e-30))


CASES = [
    # lens, hq, hk, (dqk, dv), fixed, causal, window
    ([1], 8, 2, (64, 64), True, True, None),
    ([130, 130], 6, 2, (64, 64), True, True, None),
    ([77, 1, 300, 0, 129], 8, 1, (128, 128), False, True, None),
    ([256, 511], 5, 1, (128, 128), False, False, None),
    ([400, 33], 12, 4, (192, 128), False, True, (63, 0)),
    ([200, 140], 14, 2, (64, 64), False, False, (5, 17)),
    ([384, 384], 4, 4, (128, 128), True, True, None),
    ([1000], 32, 8, (128, 128), True, True, (200, 0)),
    ([260, 129], 6, 3, (192, 128), False, True, None),
    # (the backward gives groups of few key tiles in parts; these keep them whole, or in two parts)
    ([130] * 20, 8, 4, (64, 64), True, True, None),
    ([70 + 9 * i for i in range(40)], 6, 2, (128, 128), False, True, (100, 0)),
    ([640] * 16, 4, 1, (128, 128), True, True, None),
    ([333] * 14, 8, 4, (192, 128), False, False, None),
    ([200] * 20, 4, 2, (192, 128), False, True, None),
]


def test_parts_of_the_cases():
    """The cases above have groups whole, in several parts of several heads, and of one each."""
    kinds = set()
    for lens, hq, hk, (dqk, dv), fixed, _, _ in CASES:
        B, T = len(lens), lens[0] if fixed else sum(lens)
        need = binding.attn_bwd_grouped_workspace_size(B, hq, hk, T, T, dqk, dv, not fixed)
        own = binding.attn_bwd_workspace_size(B, hq, T, T, dqk, dv, not fixed)
        parts = (need - own) // ((B * T if fixed else T) * hk * (dqk + dv) * 4)
        if hq > hk:
            kinds.add("whole" if parts == 0 else "each" if parts == hq // hk else "several")
    assert kinds == {"whole", "each", "several"}


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("det", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_backward(case, packed, det):
    lens, hq, hk, (dqk, dv), fixed, causal, window = CASES[case]
    q, k, v, dO = _inputs(case, lens, hq, hk, dqk, dv, packed, fixed)
    scale = 1.0 / math.sqrt(dqk)
    cu = None if fixed else [sum(lens[:i]) for i in range(len(lens) + 1)]
    o, lse = binding.forward(q, k, v, causal=causal, cu_seqlens=cu, window=window)
    o2, none = binding.forward(q, k, v, causal=causal, cu_seqlens=cu, window=window,
                               with_lse=False)
    assert none is None and torch.equal(o, o2)
    grads = binding.backward(q, k, v, o, dO, lse, causal=causal, cu_seqlens=cu, window=window,
                             deterministic=det)
    assert binding.attn_fwd_status() == binding.ATTN_OK
    ref = _reference(q, k, v, dO, lens, lens, scale, causal, window)
    assert _norm_err(o, ref[0]) <= TOL_O
    stat = lse.transpose(0, 1).reshape(hq, -1) if fixed else lse
    assert float((stat.double() - ref[1]).abs().max()) <= TOL_LSE
    for name, got, want, x in zip("qkv", grads, ref[2:], (q, k, v)):
        assert got.shape == x.shape
        if float(want.norm()) < 1e-9:  # rows that see one key: the gradient is zero
            assert float(got.float().norm()) <= 1e-2 * float(dO.float().norm())
        else:
            assert _norm_err(got, want) <= TOL_GRAD, name
    if det:
        again = binding.backward(q, k, v, o, dO, lse, causal=causal, cu_seqlens=cu,
                                 window=window, deterministic=True)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_against_repeated_keys():
    """The forward is the call on repeated keys bit by bit, and dk, dv are its group sums."""
    q, k, v, dO = _inputs(3, [700], 8, 2, 128, 128, False, True)
    o, lse = binding.forward(q, k, v, causal=True)
    wide = lambda t: t.repeat_interleave(4, 2).contiguous()
    ow, lw = binding.forward(q, wide(k), wide(v), causal=True)
    assert torch.equal(o, ow) and torch.equal(lse, lw)
    dq, dk, dv = binding.backward(q, k, v, o, dO, lse, causal=True, deterministic=True)
    dqw, dkw, dvw = binding.backward(q, wide(k), wide(v), o, dO, lse, causal=True,
                                     deterministic=True)
    assert torch.equal(dq, dqw)
    total = lambda t: t.unflatten(2, (2, 4)).double().sum(3)
    for got, want in ((dk, total(dkw)), (dv, total(dvw))):
        # (each summand there is rounded to bf16: 2^-9 of it at worst, summed in quadrature)
        assert _norm_err(got, want) <= 2.0 ** -7


def test_separate_key_lengths_outputs_and_streams():
    lens, lens_k = [5, 64, 0, 200], [130, 64, 7, 333]
    q, k, v, dO = _inputs(9, lens, 8, 2, 128, 128, False, False, lens_k)
    cq = [sum(lens[:i]) for i in range(5)]
    ck = [sum(lens_k[:i]) for i in range(5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = binding.forward(q, k, v, causal=True, cu_seqlens=cq, cu_seqlens_k=ck, stream=side)
    buf = torch.full((sum(lens_k), 2 * 128 * 2 + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    dk = buf[:, :256].unflatten(1, (2, 128))
    dv = buf[:, 256:512].unflatten(1, (2, 128))
    dq = torch.empty_like(q)
    with torch.cuda.stream(side):
        got = binding.backward(q, k, v, o, dO, lse, causal=True, cu_seqlens=cq, cu_seqlens_k=ck,
                               out=(dq, dk, dv))
    torch.cuda.synchronize()
    assert got[0] is dq and got[1] is dk
    ref = _reference(q, k, v, dO, lens, lens_k, 1 / math.sqrt(128), True, None)
    assert _norm_err(o, ref[0]) <= TOL_O
    for a, b in zip(got, ref[2:]):
        assert _norm_err(a, b) <= TOL_GRAD
    assert (dk[194:201] == 0).all() and (dv[194:201] == 0).all()  # keys without queries
    assert (buf[:, 512:] == 7).all()


def test_captured_step():
    q, k, v, dO = _inputs(4, [300], 8, 2, 128, 128, False, True)
    o, lse = binding.forward(q, k, v, causal=True)
    want = binding.backward(q, k, v, o, dO, lse, causal=True, deterministic=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = binding.forward(q, k, v, causal=True)
        got = binding.backward(q, k, v, og, dO, lg, causal=True, deterministic=True)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(og, o) and all(torch.equal(a, b) for a, b in zip(got, want))
