"""Local windows longer than the sequence, up to the largest integer: they see what a window
of the sequence's length sees."""
import pytest
import torch

from attention_backward_flashattention_gb300 import binding

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


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("d", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("window,same", [((BIG, 0), (700, 0)), ((BIG, BIG), (700, 700)),
                                         ((40, BIG), (40, 700)), ((-1, BIG), (-1, 700)),
                                         ((2 ** 30, 3), (700, 3)), ((BIG - 600, 0), (700, 0))])
@pytest.mark.parametrize("varlen", [False, True])
def test_windows_of_any_length(d, window, same, varlen):
    dqk, dv = d
    H, Tq, Tk = 2, 300, 700
    q, k, v, dO = (_rand(i, 1, T, H, w) for i, (T, w) in
                   enumerate([(Tq, dqk), (Tk, dqk), (Tk, dv), (Tq, dv)]))
    kw = {}
    if varlen:
        q, k, v, dO = q[0], k[0], v[0], dO[0]
        kw = dict(cu_seqlens=[0, 130, 300], cu_seqlens_k=[0, 401, 700])
    got, want = [], []
    for w, dst in ((same, want), (window, got)):
        o, lse = binding.forward(q, k, v, window=w, **kw)
        grads = binding.backward(q, k, v, o, dO, lse, window=w, deterministic=True, **kw)
        dst.extend([o, lse, *grads])
    assert binding.attn_fwd_status() == binding.ATTN_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(t.count_nonzero() > 0 for t in want)
