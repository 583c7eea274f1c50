"""Norms of heads, their gradients and the append over thousands of token rows, where a block has
several tokens at a time (and in the gradient several chunks one after the other), against the formulas
in fp64."""
import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests import test_gpu_norm as small
from tests.paged_common import BF16_HALF, inv_freq, rotate64

pytestmark = pytest.mark.gpu
EPS = small.EPS


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _groups(d):
    """Heads side by side in a block."""
    return {64: 64, 128: 32, 192: 16}[d]


def _most(dim):
    return min(32, 2048 // (dim // 2)) if dim else 32


def norm_chunk(rows, H, d, dim):
    """Token rows of a chunk (the library's rule, to see that a case has several)."""
    tokens = min(max(1, 16 * _groups(d) // H), _most(dim))
    while tokens > 1 and -(-rows // tokens) < 4 * _sms():
        tokens //= 2
    return tokens


def append_chunk(T, heads, d, dim):
    tokens = max(1, 8 * _groups(d) // heads)
    while tokens > 1 and T // tokens < 4 * _sms():
        tokens //= 2
    return min(tokens, _most(dim))


# d, Hq, Hk, begin, dim, interleaved, (B, T) or lengths of queries and of keys, pos0,
# whether the queries' gradient has more chunks than blocks
CASES = [
    (64, 12, 4, 0, 64, False, (2, 2500), 7, False),
    (64, 1, 2, 0, 32, True, (1, 40000), 0, True),
    (128, 32, 8, 0, 128, False, (1, 20000), 1000003, True),
    (128, 4, 4, 0, 0, False, (3, 1700), 0, False),
    (128, 6, 3, 64, 64, True, ([1, 0, 700, 3, 1501, 9, 2000, 1], None), 5, True),
    (128, 6, 2, 0, 128, False, ([1, 0, 700, 3, 1501, 2000], [40, 3, 701, 900, 1501, 2077]), 0, True),
    (192, 5, 3, 128, 64, True, ([600] * 9 + [33], None), 0, False),
    (192, 2, 1, 0, 192, False, (2, 20000), 3, True),
]


def _offsets(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_norm_and_gradients(case):
    d, hq, hk, begin, dim, inter, shape, pos0, wraps = CASES[case]
    g = torch.Generator(device="cpu").manual_seed(100 + case)
    packed = isinstance(shape[0], list)
    if packed:
        lq, lk = shape[0], shape[1] or shape[0]
        rq, rk = (sum(lq),), (sum(lk),)
        cu = {"cu_seqlens": _offsets(lq)}
        if shape[1]:
            cu["cu_seqlens_k"] = _offsets(lk)
        # the queries are the last positions of their sequence's keys
        pq = torch.cat([torch.arange(m - n, m) for n, m in zip(lq, lk)]).cuda() + pos0
        pk = torch.cat([torch.arange(m) for m in lk]).cuda() + pos0
    else:
        rq = rk = shape
        cu = {}
        pq = pk = torch.arange(shape[1]).repeat(shape[0]).cuda() + pos0
    together = small._slices(g, rq, (hq, hk), d)[:2] if rq == rk else \
        [small._rand(g, *rq, hq, d), small._rand(g, *rk, hk, d)]
    rows = [t.numel() // (t.shape[-1] * t.shape[-2]) for t in together]
    sizes = [norm_chunk(n, h, d, dim) for n, h in zip(rows, (hq, hk))]
    assert min(sizes) > 1 and (-(-rows[0] // sizes[0]) > 1024) == wraps
    w = [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    freq = inv_freq(dim) if dim else None
    rot = binding.Rotation(freq, begin=begin, interleaved=inter) if dim else None
    norm = binding.HeadNorm(*w, eps=EPS)
    flat = lambda t: t.reshape(-1, *t.shape[-2:])

    got = binding.norm_rope(*together, norm, rot, pos0=pos0, **cu)
    for y, x, v, pos in zip(got, together, w, (pq, pk)):
        ref, tol = small.forward64(flat(x), v, pos, freq, begin, inter)
        assert ((flat(y).double() - ref).abs() <= tol).all()

    dy = [small._rand(g, *t.shape) for t in together]
    out = binding.norm_rope_backward(*together, *dy, norm, rot, pos0=pos0, **cu)
    again = binding.norm_rope_backward(*together, *dy, norm, rot, pos0=pos0, **cu)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    for i, (x, e, v, pos) in enumerate(zip(together, dy, w, (pq, pk))):
        leaf = flat(x).double().requires_grad_()
        wl = v.double().requires_grad_()
        y = small.normed64(leaf, wl)
        if freq is not None:
            y = rotate64(y, pos, freq, begin, inter)[0]
        y.backward(flat(e).double())
        with torch.no_grad():
            # (the bounds of an element: tests/test_gpu_norm.py)
            x64 = leaf.detach()
            r = torch.rsqrt(x64.square().mean(-1, keepdim=True) + EPS)
            gm = flat(e).double().abs()
            if freq is not None:
                gm = torch.maximum(gm, rotate64(flat(e), pos, freq, begin, inter, -1.0)[1])
            gw = gm * wl.abs()
            mag = r * (gw + x64.abs() * r * r * (gw * x64.abs()).mean(-1, keepdim=True))
            tol = BF16_HALF * leaf.grad.abs() + 2.0 ** -14 * mag * (1 + BF16_HALF)
            assert ((flat(out[i]).double() - leaf.grad).abs() <= tol).all()
            # A weight's gradient: terms off by 2^-17 each; a lane adds the heads of its chunks, 17 of
            # each at most, then come a warp's lanes (3), eight warps, and 1024 rows by eight slices of
            # 16 warps (8 rows each, 16 and 8 sums): each addition is off by 2^-24 of the sum of
            # absolute terms.
            chunks = -(-(-(-rows[i] // sizes[i])) // 1024)
            depth = 17 * chunks + 3 + 8 + 8 + 16 + 8
            tol = (gm * x64.abs() * r).sum((0, 1)) * (2.0 ** -17 + depth * 2.0 ** -24)
            assert ((out[2 + i].double() - wl.grad).abs() <= tol).all()


@pytest.mark.parametrize("kind,order", [("bf16", "token"), ("bf16", "head"), ("e4m3", "token")])
@pytest.mark.parametrize("d,begin,dim,inter", [((64, 64), 0, 64, False), ((128, 128), 0, 64, True),
                                               ((192, 128), 128, 64, True),
                                               ((128, 128), 0, 0, False)])
@pytest.mark.parametrize("new,lens", [
    ([1, 2500, 0, 7, 3001, 4, 491], [1, 2600, 9, 7, 4000, 2, 500]), ([4000] * 5, [4000] * 4 + [4321])])
def test_append_of_prompts(d, begin, dim, inter, kind, order, new, lens):
    """Sequences' borders inside a block's tokens, and one that brings more tokens than it has."""
    assert append_chunk(sum(new), 9, d[0], dim) > 1
    small.test_append(d, begin, dim, inter, kind, order, new, lens)
