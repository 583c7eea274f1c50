"""Norm of query and key heads with the rotation, its gradient, and the append with both, against
the formulas in fp64."""
import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import (BF16_HALF, E4M3_HALF, bits, inv_freq, make_cache, make_table,
                                nan_bits, rotate64)

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()


def normed64(x, w):
    x = x.double()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return y if w is None else y * w.double()


def forward64(x, w, pos, freq, begin, inter):
    """y and a bound of its error: the sum of d squares rounds at 2^-24 each (d/2 of that in r),
    rsqrt and the products at 2^-22: below 2^-16 of |a| + |b| with the rotation's 2^-20; and one
    rounding to bf16."""
    n = normed64(x, w)
    if freq is None:
        y, mag = n, n.abs()
    else:
        y, mag = rotate64(n, pos, freq, begin, inter)
        mag = torch.maximum(mag, n.abs())
    return y, BF16_HALF * y.abs() + 2.0 ** -16 * mag * (1 + BF16_HALF)


def _rand(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def _slices(g, rows, heads, d):
    x = _rand(g, *rows, (sum(heads) + 1) * d)
    parts = x.split([h * d for h in heads] + [d], -1)
    return [p.unflatten(-1, (h, d)) for p, h in zip(parts, heads)]


def _positions(B, T, lens, pos0, shift=0):
    if lens is None:
        return (torch.arange(T).cuda() + pos0 + shift).repeat(B)
    return torch.cat([torch.arange(n) for n in lens]).cuda() + pos0


CASES = [
    # d, Hq, Hk, begin, dim (0: no rotation), interleaved, B, T or lens, pos0
    (64, 1, 1, 0, 64, False, 1, 1, 0),
    (64, 12, 4, 0, 32, True, 2, 65, 7),
    (128, 32, 8, 0, 128, False, 2, 130, 0),
    (128, 5, 1, 0, 128, True, 3, [1, 0, 300], 1000003),
    (192, 16, 3, 128, 64, True, 1, 77, 0),
    (192, 7, 7, 0, 192, False, 2, [40, 2], 5),
    (128, 70, 2, 64, 64, False, 1, 3, 0),
    (128, 4, 4, 0, 0, False, 4, 33, 0),
]


def _case(i):
    d, hq, hk, begin, dim, inter, B, T, pos0 = CASES[i]
    lens = T if isinstance(T, list) else None
    g = torch.Generator(device="cpu").manual_seed(i)
    rows = (sum(lens),) if lens else (B, T)
    q, k = _slices(g, rows, (hq, hk), d)
    wq = (1 + 0.3 * torch.randn(d, generator=g)).cuda()
    wk = (1 + 0.3 * torch.randn(d, generator=g)).cuda() if i % 2 else None
    freq = inv_freq(dim) if dim else None
    rot = binding.Rotation(freq, begin=begin, interleaved=inter) if dim else None
    cu = None if lens is None else [sum(lens[:j]) for j in range(len(lens) + 1)]
    pos = _positions(B, T, lens, pos0)
    return d, q, k, wq, wk, freq, begin, inter, rot, cu, pos, pos0, g


@pytest.mark.parametrize("case", range(len(CASES)))
def test_norm_rope(case):
    d, q, k, wq, wk, freq, begin, inter, rot, cu, pos, pos0, g = _case(case)
    norm = binding.HeadNorm(wq, wk, eps=EPS)
    got = binding.norm_rope(q, k, norm, rot, pos0=pos0, cu_seqlens=cu)
    for y, x, w in zip(got, (q, k), (wq, wk)):
        ref, tol = forward64(x.reshape(-1, *x.shape[-2:]), w, pos, freq, begin, inter)
        assert ((y.double().reshape(ref.shape) - ref).abs() <= tol).all()
    # each alone, in place, on another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i, x in enumerate((q, k)):
        mine = x.clone() if x.is_contiguous() else x
        keep = x.clone()
        args = (mine, None) if i == 0 else (None, mine)
        one = binding.norm_rope(*args, norm, rot, pos0=pos0, cu_seqlens=cu, out=args, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(one[i], got[i]) and one[1 - i] is None
        mine.copy_(keep)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_norm_rope_backward(case):
    d, q, k, wq, wk, freq, begin, inter, rot, cu, pos, pos0, g = _case(case)
    norm = binding.HeadNorm(wq, wk, eps=EPS)
    dyq, dyk = _rand(g, *q.shape), _rand(g, *k.shape)
    dq, dk, dqw, dkw = binding.norm_rope_backward(q, k, dyq, dyk, norm, rot, pos0=pos0,
                                                  cu_seqlens=cu)
    again = binding.norm_rope_backward(q, k, dyq, dyk, norm, rot, pos0=pos0, cu_seqlens=cu)
    assert torch.equal(dqw, again[2]) and (dkw is None) == (wk is None)
    for dx, dw, x, dy, w in ((dq, dqw, q, dyq, wq), (dk, dkw, k, dyk, wk)):
        flat = lambda t: t.reshape(-1, *t.shape[-2:])
        leaf = flat(x).double().requires_grad_()
        wl = (torch.ones(d).cuda() if w is None else w).double().requires_grad_()
        y = normed64(leaf, wl)
        if freq is not None:
            y = rotate64(y, pos, freq, begin, inter)[0]
        y.backward(flat(dy).double())
        # bounds: g = w R^T dy is off by 2^-20 of |a| + |b|; both sums by d 2^-24 of their absolute
        # terms, r by 2^-17: in all below 2^-14 of r (|g| + |x| r^2 mean |g x|)
        x64 = flat(x).double()
        r = torch.rsqrt(x64.square().mean(-1, keepdim=True) + EPS)
        gm = flat(dy).double().abs()
        if freq is not None:
            gm = torch.maximum(gm, rotate64(flat(dy), pos, freq, begin, inter, -1.0)[1])
        gw = gm * wl.abs()
        mag = r * (gw + x64.abs() * r * r * (gw * x64.abs()).mean(-1, keepdim=True))
        tol = BF16_HALF * leaf.grad.abs() + 2.0 ** -14 * mag * (1 + BF16_HALF)
        assert ((flat(dx).double() - leaf.grad).abs() <= tol.detach()).all()
        if dw is not None:
            n = x64.shape[0] * x64.shape[1]
            tol = (gm * x64.abs() * r).sum((0, 1)) * (2.0 ** -17 + n * 2.0 ** -24)
            assert ((dw.double() - wl.grad).abs() <= tol).all()
    # over its own inputs
    keep = q.clone()
    out = binding.norm_rope_backward(q, k, dyq, dyk, norm, rot, pos0=pos0, cu_seqlens=cu,
                                     out=(dyq, dyk))
    assert torch.equal(out[0], dq) and torch.equal(dyk, dk) and torch.equal(q, keep)


def test_gradient_formula_against_differences():
    """dx and dw of the definition by autograd (what the test above holds the kernel to), by
    central differences."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 64, generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(64, generator=g, dtype=torch.float64)
    pos, dy = torch.arange(2), torch.randn(2, 3, 64, generator=g, dtype=torch.float64)
    loss = lambda a, b: (rotate64(normed64(a, b), pos, inv_freq(64), 0, False)[0] * dy).sum()
    xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
    loss(xl, wl).backward()
    h = 1e-6
    for t, grad in ((x, xl.grad), (w, wl.grad)):
        for i in range(0, t.numel(), 7):
            e = torch.zeros(t.numel(), dtype=torch.float64)
            e[i] = h
            e = e.view(t.shape)
            at = lambda s: loss(x + s * e, w) if t is x else loss(x, w + s * e)
            assert abs((at(1) - at(-1)) / (2 * h) - grad.view(-1)[i]) <= 1e-7


def test_rows_of_zeros_and_extremes():
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    x[0, 1] = 1e-30
    x[0, 2] = 1e18
    x[0, 3, 0] = float("nan")
    norm = binding.HeadNorm(eps=1e-6)
    y, _ = binding.norm_rope(x, None, norm)
    assert (y[0, 0] == 0).all() and torch.isfinite(y[0, 1]).all()
    assert (y[0, 2].float() - 1).abs().max() <= 2.0 ** -8
    assert torch.isnan(y[0, 3, 0]).all() and (y[0, 3, 1] == 0).all()


def test_captured_step():
    """Norms and their gradients in a graph, replayed, have the bits of the calls in turn."""
    g = torch.Generator().manual_seed(2)
    q, k, dq, dk = (_rand(g, 2, 700, h, 128) for h in (8, 2, 8, 2))
    w = torch.rand(128, generator=g).cuda() + 0.5
    norm, rot = binding.HeadNorm(w, w, EPS), binding.Rotation(inv_freq(128))
    call = lambda: (*binding.norm_rope(q, k, norm, rot),
                    *binding.norm_rope_backward(q, k, dq, dk, norm, rot))
    want = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for t in got:
        t.fill_(7)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_weights_that_move():
    """A parameter whose memory is replaced: the next call reads the new one."""
    x = torch.randn(1, 5, 2, 64, device="cuda").to(torch.bfloat16)
    w = torch.nn.Parameter(torch.ones(64, device="cuda"))
    norm = binding.HeadNorm(w, None)
    one, _ = binding.norm_rope(x, None, norm)
    w.data = torch.full((64,), 2.0, device="cuda")
    two, _ = binding.norm_rope(x, None, norm)
    assert torch.equal(two, one * 2)


def test_append_keys_alone():
    page, heads, d = 16, 3, 128
    g = torch.Generator().manual_seed(1)
    table, pages = make_table([40, 7], page, 3)
    caches = [(make_cache(pages, page, heads, d, "bf16", "token", 4),
               make_cache(pages, page, heads, d, "bf16", "token", 5)) for _ in range(2)]
    lens = torch.tensor([40, 7], dtype=torch.int32).cuda()
    q, k, v = (_rand(g, 10, h, d) for h in (6, heads, heads))
    norm, rot = binding.HeadNorm(eps=EPS), binding.Rotation(inv_freq(d))
    none = binding.cache_append(binding.PagedCache(*caches[0]), k, v, table, lens, rotation=rot,
                                norm=norm)
    binding.cache_append(binding.PagedCache(*caches[1]), k, v, table, lens, q=q, rotation=rot,
                         norm=norm)
    assert none is None
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    assert binding.attn_cache_status() == binding.ATTN_OK


@pytest.mark.parametrize("kind,order", [("bf16", "token"), ("bf16", "head"), ("e4m3", "token")])
@pytest.mark.parametrize("d,begin,dim,inter", [((64, 64), 0, 64, False), ((128, 128), 0, 64, True),
                                               ((192, 128), 128, 64, True),
                                               ((128, 128), 0, 0, False)])
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [5, 0, 33]), ([40, 0, 3], [40, 9, 100]),
                                      ([200, 5], [300, 3])])
def test_append(d, begin, dim, inter, kind, order, new, lens):
    dqk, dv = d
    heads, Hq, page = 3, 6, 16
    g = torch.Generator(device="cpu").manual_seed(dqk + len(new))
    table, pages = make_table(lens, page, 3)
    kc = make_cache(pages, page, heads, dqk, kind, order, 4)
    vc = make_cache(pages, page, heads, dv, kind, order, 5)
    before = bits(kc).clone(), bits(vc).clone()
    unit = (1 + torch.rand(heads, generator=g)).cuda() / 64 if kind == "e4m3" else None
    cache = binding.PagedCache(kc, vc, unit, unit)
    T = sum(new)
    q, k, v = _rand(g, T, Hq, dqk), _rand(g, T, heads, dqk), _rand(g, T, heads, dv)
    wq, wk = ((1 + 0.3 * torch.randn(dqk, generator=g)).cuda() for _ in range(2))
    norm = binding.HeadNorm(wq, wk, eps=EPS)
    freq = inv_freq(dim) if dim else None
    rot = binding.Rotation(freq, begin=begin, interleaved=inter) if dim else None
    cu = None if len(set(new)) == 1 else [sum(new[:i]) for i in range(len(new) + 1)]
    lens_d = torch.tensor(lens, dtype=torch.int32).cuda()
    q_out = torch.full_like(q, 3.0)
    got = binding.cache_append(cache, k, v, table, lens_d, q=q, rotation=rot, cu_seqlens=cu,
                               q_out=q_out, norm=norm)
    assert got is q_out and binding.attn_cache_status() == binding.ATTN_OK
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
    ends = torch.tensor([sum(new[:i + 1]) for i in range(len(new))]).cuda()
    pos = lens_d.long()[seq] - (ends[seq] - torch.arange(T).cuda())
    live = pos >= 0
    ref, tol = forward64(q, wq, pos, freq, begin, inter)
    assert ((got.double() - ref).abs() <= tol)[live].all() and (got[~live] == 3).all()
    at = (table[seq, pos.clamp(min=0) // page].long()[live], pos[live] % page)
    if cu is not None and all(m >= n for m, n in zip(lens, new)):  # the bits that norm_rope gives
        shift = [m - n for m, n in zip(lens, new)]
        for b in range(len(new)):
            r = slice(cu[b], cu[b + 1])
            if r.stop > r.start:
                one, key = binding.norm_rope(q[None, r], k[None, r], norm, rot, pos0=shift[b])
                assert torch.equal(got[r], one[0])
                if kind == "bf16":
                    j = torch.arange(shift[b], lens[b]).cuda()
                    assert torch.equal(kc[table[b].long()[j // page], j % page], key[0])
    rk, tk = forward64(k, wk, pos, freq, begin, inter)
    for c, want, tol, raw in ((kc, rk, tk, before[0]), (vc, v.double(), None, before[1])):
        have = bits(c)[at].view(c.dtype).double()
        want = want[live]
        if kind == "bf16":
            limit = 0 if tol is None else tol[live]
        else:
            # rounding to e4m3 (half a step, at least of a subnormal, 2^-10) of a value that is off
            # by what the norm is
            u = unit.double()[:, None]
            have, off = have * u, 0 if tol is None else tol[live]
            limit = E4M3_HALF * want.abs() + 2.0 ** -10 * u + 2 * off
            want = want.clamp(min=(-448 * u), max=(448 * u))
        assert ((have - want).abs() <= limit).all()
        same = torch.ones(c.shape[:2], dtype=torch.bool, device="cuda")
        same[at] = False
        assert torch.equal(bits(c)[same], raw[same])
