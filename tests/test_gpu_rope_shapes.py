"""attn_rope where a thread walks over several rows or several units of a row, and where its
angles lie next to a zero of the sine or the cosine."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import BF16_HALF, inv_freq, rotate64, rotation_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()


def _rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _check(got, x, pos, freq, begin, inter, sign=1.0):
    for b in range(x.shape[0]):
        for lo in range(0, x.shape[1], 4096):
            rows = slice(lo, lo + 4096)
            want, mag = rotate64(x[b, rows], pos[rows], freq, begin, inter, sign)
            over = (got[b, rows].double() - want).abs() - rotation_bound(want, mag)
            assert (over <= 0).all(), f"sequence {b}, rows from {lo}: over by {over.max()}"


@pytest.mark.parametrize("d,begin,dim", [(64, 0, 64), (128, 32, 64), (128, 0, 128),
                                         (192, 128, 64)])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hk", [
    (2, 12001, 12003, 16, 4),   # several rows a thread, for queries and keys of other widths
    (1, 41003, 41003, 4, 1),    # many rows side by side
    (1, 5001, 5001, 40, 1),     # rows of more units than a block has threads (d 128, 192)
    (1, 3, 5003, 1, 72)])       # and where the keys' blocks are the wide ones
@pytest.mark.parametrize("inverse", [False, True])
def test_long_and_wide(d, begin, dim, B, Tq, Tk, Hq, Hk, inverse):
    q, k = _rand(1, B, Tq, Hq, d), _rand(2, B, Tk, Hk, d)
    freq, inter = inv_freq(dim), inverse
    rot = binding.Rotation(freq, begin=begin, interleaved=inter)
    qo, ko = binding.rope(q, k, rot, inverse=inverse, pos0=7)
    sign = -1.0 if inverse else 1.0
    _check(qo, q, torch.arange(Tq).cuda() + 7 + Tk - Tq, freq, begin, inter, sign)
    _check(ko, k, torch.arange(Tk).cuda() + 7, freq, begin, inter, sign)


def test_long_variable_length():
    lens = [9000, 1, 0, 13007, 300]
    cu = [sum(lens[:i]) for i in range(6)]
    q, k = _rand(3, cu[-1], 8, 128), _rand(4, cu[-1], 2, 128)
    freq = inv_freq(128)
    qo, ko = binding.rope(q, k, binding.Rotation(freq), cu_seqlens=cu)
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    _check(qo[None], q[None], pos, freq, 0, False)
    _check(ko[None], k[None], pos, freq, 0, False)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_angles_next_to_a_zero_of_the_sine_or_the_cosine(inter, inverse):
    """A quarter, a half, three quarters of a turn and a whole one, a little more or less: the
    small one of sine and cosine has as many right bits as the large one."""
    freq = [math.pi / 2 * k * (1 + sgn * 1.3906 * 2.0 ** -e) for k in (1, 2, 3, 4)
            for sgn in (-1, 1) for e in (15, 17, 19, 21)]
    dim = 2 * len(freq)
    rot = binding.Rotation(freq, interleaved=inter)
    ia = torch.arange(0, dim, 2) if inter else torch.arange(dim // 2)
    ib = ia + (1 if inter else dim // 2)
    q = torch.zeros(1, 2, 2, dim, dtype=torch.bfloat16)
    q[:, :, 0, ia] = 1.0   # (cos, sin)
    q[:, :, 1, ib] = 1.0   # (-sin, cos)
    q = q.cuda()
    got, _ = binding.rope(q, None, rot, inverse=inverse)
    want, _ = rotate64(q[0], torch.arange(2).cuda(), freq, 0, inter, -1.0 if inverse else 1.0)
    # beside the rounding to bf16: an angle's distance from the nearest quarter turn is rounded
    # to fp32 (2^-24 of it) and held to 2^-33 of a half turn (below 2^-31); sincospi is good to
    # 2^-22 of its value
    bound = (BF16_HALF + 2.0 ** -21) * want.abs() + 2.0 ** -31
    over = (got[0].double() - want).abs() - bound
    assert (over <= 0).all(), f"over by {over.max()}"
