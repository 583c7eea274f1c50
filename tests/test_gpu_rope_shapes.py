"""attn_rope where its angles lie next to a zero of the sine or the cosine."""
import math

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import BF16_HALF, rotate64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()


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
