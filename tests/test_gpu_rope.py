"""attn_rope on the GPU against the rotation in 64 bits: styles, partly rotated heads,
layouts, lengths, far positions, in place, and the gradient."""
import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import inv_freq, rotate64, rotation_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()


def _rand(seed, *shape):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def _check(got, x, pos, freq, begin, inter, sign=1.0):
    want, mag = rotate64(x.reshape(-1, *x.shape[-2:]), pos, freq, begin, inter, sign)
    got = got.reshape(want.shape)
    over = (got.double() - want).abs() - rotation_bound(want, mag)
    assert (over <= 0).all(), f"over by {over.max()}"
    still = torch.ones(x.shape[-1], dtype=torch.bool)
    still[begin:begin + 2 * len(freq)] = False
    assert torch.equal(got[..., still], x.reshape(want.shape)[..., still])


@pytest.mark.parametrize("d,begin,dim", [(64, 0, 64), (64, 0, 32), (64, 32, 16), (128, 0, 128),
                                         (128, 16, 96), (192, 128, 64), (192, 0, 192)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hk", [(1, 1, 1, 1, 1), (2, 7, 7, 3, 2), (3, 33, 50, 5, 1)])
def test_fixed_length(d, begin, dim, inter, B, Tq, Tk, Hq, Hk):
    q, k = _rand(1, B, Tq, Hq, d), _rand(2, B, Tk, Hk, d)
    freq = inv_freq(dim)
    rot = binding.Rotation(freq, begin=begin, interleaved=inter)
    qo, ko = binding.rope(q, k, rot)
    # the queries are the last Tq positions of the keys
    _check(qo, q, (torch.arange(Tq).cuda() + Tk - Tq).repeat(B), freq, begin, inter)
    _check(ko, k, torch.arange(Tk).cuda().repeat(B), freq, begin, inter)


@pytest.mark.parametrize("pos0", [0, 65537, 1000003, 2147483647 - 300])
def test_far_positions(pos0):
    q = _rand(3, 1, 300, 2, 128)
    freq = inv_freq(128)
    qo, none = binding.rope(q, None, binding.Rotation(freq), pos0=pos0)
    assert none is None
    # the angle in fp64 is itself off by pos * 2^-53 at most: 2^-22 at 2^31
    want, mag = rotate64(q[0], torch.arange(300).cuda() + pos0, freq, 0, False)
    over = (qo[0].double() - want).abs() - rotation_bound(want, mag) - 2.0 ** -53 * pos0 * mag
    assert (over <= 0).all()


def test_more_queries_than_keys_turn_backwards():
    q, k = _rand(4, 1, 9, 2, 64), _rand(5, 1, 4, 2, 64)
    freq = inv_freq(64)
    qo, _ = binding.rope(q, k, binding.Rotation(freq))
    _check(qo, q, torch.arange(9).cuda() - 5, freq, 0, False)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("varlen", [False, True])
def test_keys_beside_no_queries(varlen, given):
    """A step without queries still turns its keys."""
    q, k, freq = _rand(40, 1, 0, 2, 64), _rand(41, 1, 7, 2, 64), inv_freq(64)
    kw = {}
    if varlen:
        q, k, kw = q[0], k[0], dict(cu_seqlens=[0, 0, 0], cu_seqlens_k=[0, 3, 7])
    if given:
        kw["out"] = (torch.empty_like(q), torch.full_like(k, 7.0))
    qo, ko = binding.rope(q, k, binding.Rotation(freq), **kw)
    assert qo.shape == q.shape
    pos = [0, 1, 2, 0, 1, 2, 3] if varlen else range(7)
    _check(ko, k, torch.tensor(list(pos)).cuda(), freq, 0, False)


def test_one_side_of_a_variable_length_pair():
    """Queries without their keys, and keys without their queries, at the pair's positions."""
    cu, cuk = [0, 2, 2, 7], [0, 6, 9, 14]
    q, k, rot = _rand(42, 7, 3, 64), _rand(43, 14, 2, 64), binding.Rotation(inv_freq(64))
    qo, ko = binding.rope(q, k, rot, cu_seqlens=cu, cu_seqlens_k=cuk)
    pos = torch.tensor([4, 5, 0, 1, 2, 3, 4]).cuda()
    _check(qo, q, pos, inv_freq(64), 0, False)
    q1, none = binding.rope(q, None, rot, cu_seqlens=cu, cu_seqlens_k=cuk)
    assert none is None and torch.equal(q1, qo)
    none, k1 = binding.rope(None, k, rot, cu_seqlens=cu, cu_seqlens_k=cuk)
    assert none is None and torch.equal(k1, ko)


@pytest.mark.parametrize("inter", [False, True])
def test_variable_length(inter):
    lq, lk = [5, 0, 1, 130, 17], [9, 3, 1, 130, 40]
    cq = [sum(lq[:i]) for i in range(6)]
    ck = [sum(lk[:i]) for i in range(6)]
    q, k = _rand(6, sum(lq), 4, 192), _rand(7, sum(lk), 2, 192)
    freq = inv_freq(64)
    rot = binding.Rotation(freq, begin=128, interleaved=inter)
    qo, ko = binding.rope(q, k, rot, cu_seqlens=cq, cu_seqlens_k=ck, pos0=11)
    pq = torch.cat([torch.arange(a) + b - a for a, b in zip(lq, lk)]).cuda() + 11
    pk = torch.cat([torch.arange(b) for b in lk]).cuda() + 11
    _check(qo, q, pq, freq, 128, inter)
    _check(ko, k, pk, freq, 128, inter)


def test_packed_in_place_leaves_the_values_slot():
    qkv = _rand(8, 2, 37, 3, 12, 64)
    before = qkv.clone()
    freq = inv_freq(64)
    rot = binding.Rotation(freq)
    q, k = qkv.select(2, 0), qkv.select(2, 1)
    binding.rope(q, k, rot, out=(q, k))
    assert torch.equal(qkv.select(2, 2), before.select(2, 2))
    pos = torch.arange(37).cuda().repeat(2)
    _check(q, before.select(2, 0), pos, freq, 0, False)
    _check(k, before.select(2, 1), pos, freq, 0, False)
    out = binding.rope(before.select(2, 0), before.select(2, 1), rot)
    assert torch.equal(out[0], q) and torch.equal(out[1], k)


def test_rows_outside_the_tensor_are_untouched():
    buf = _rand(9, 1, 40, 6, 64)
    before = buf.clone()
    part = buf[:, 8:30, :4]  # 4 of 6 heads, rows 8 .. 29
    binding.rope(part, None, binding.Rotation(inv_freq(64)), out=(part, None))
    assert torch.equal(buf[:, :8], before[:, :8]) and torch.equal(buf[:, 30:], before[:, 30:])
    assert torch.equal(buf[:, :, 4:], before[:, :, 4:])
    _check(part, before[:, 8:30, :4], torch.arange(22).cuda(), inv_freq(64), 0, False)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient(inter):
    """The inverse is the gradient: against the formula, and <dy, rope(x + e)> - <dy, rope(x)>
    = <inverse(dy), e> for the linear map, in sums of the bf16 outputs."""
    x, dy = _rand(10, 1, 64, 2, 128), _rand(11, 1, 64, 2, 128)
    freq = inv_freq(128)
    rot = binding.Rotation(freq, interleaved=inter)
    pos = torch.arange(64).cuda()
    dx, _ = binding.rope(dy, None, rot, inverse=True)
    _check(dx, dy, pos, freq, 0, inter, sign=-1.0)
    # differences: rope is linear, so a step of any size does
    for seed in range(3):
        e = _rand(20 + seed, 1, 64, 2, 128)
        xe = (x.float() + e.float()).to(torch.bfloat16)
        step = xe.double() - x.double()
        y0, y1 = (binding.rope(t, None, rot)[0].double() for t in (x, xe))
        left = (dy.double() * (y1 - y0)).sum()
        right = (dx.double() * step).sum()
        # each of y0, y1, dx is off by its rounding and fp32 arithmetic
        slack = 0.0
        for t, w in ((x, dy), (xe, dy)):
            y, m = rotate64(t[0], pos, freq, 0, inter)
            slack += (rotation_bound(y, m) * w[0].double().abs()).sum()
        y, m = rotate64(dy[0], pos, freq, 0, inter, -1.0)
        slack += (rotation_bound(y, m) * step[0].abs()).sum()
        assert abs(left - right) <= slack


@pytest.mark.parametrize("shape", [(3, 5), (7, 2, 64), (2, 3, 4, 64), (1, 1, 1), (0, 4, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_new_outputs_are_like_torch_empty(shape, dtype):
    want = torch.empty(shape, dtype=dtype, device="cuda")
    for got in (binding._empty(shape, dtype, want.device),
                binding._empty(torch.Size(shape), dtype, want.device)):
        assert got.shape == want.shape and got.stride() == want.stride()
        assert got.dtype == dtype and got.device == want.device and got.is_contiguous()
        assert not got.requires_grad
    with torch.inference_mode():
        assert binding._empty(shape, dtype, want.device).is_inference()


def test_pass_through_bits():
    """Columns that do not turn keep their bits, NaN payloads and infinities among them, and do
    not touch the others."""
    q = _rand(12, 1, 5, 2, 64)
    q[..., 32:] = float("nan")
    q[0, 1, 0, 40] = float("inf")
    out, _ = binding.rope(q, None, binding.Rotation(inv_freq(32)))
    raw = lambda t: t.contiguous().view(torch.int16)
    assert torch.equal(raw(out[..., 32:]), raw(q[..., 32:]))
    assert torch.isfinite(out[..., :32].float()).all()


def test_another_stream_and_a_captured_call():
    q, k = _rand(13, 1, 100, 4, 128), _rand(14, 1, 100, 4, 128)
    rot = binding.Rotation(inv_freq(128))
    want = binding.rope(q, k, rot)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = binding.rope(q, k, rot, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = (torch.zeros_like(q), torch.zeros_like(k))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.rope(q, k, rot, out=out)
    q.copy_(_rand(15, 1, 100, 4, 128))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], binding.rope(q, k, rot)[0]) and torch.equal(out[1], want[1])
