"""Rotation, paged cache and decode: edges that are decided on the host (no GPU needed)."""
import types

import pytest
import torch

from attention_backward_flashattention_gb300 import binding

TOP, LOW = 2 ** 31 - 1, -2 ** 31


@pytest.fixture
def seen(monkeypatch):
    """The arguments with which the library's functions are called, instead of the calls."""
    calls = {}
    names = ("attn_decode", "attn_rope", "attn_fwd_ex", "attn_bwd_ex", "attn_fwd_window",
             "attn_bwd_window")
    fake = types.SimpleNamespace(**{
        n: (lambda *a, n=n: calls.__setitem__(n, a) or 0) for n in names})
    monkeypatch.setattr(binding, "load", lambda: fake)
    return calls


@pytest.mark.parametrize("given,taken", [(5, 5), (-1, -1), (TOP, TOP), (2 ** 31, TOP),
                                         (2 ** 32, TOP), (2 ** 32 + 3, TOP), (2 ** 70, TOP),
                                         (LOW, LOW), (LOW - 1, LOW), (-2 ** 32 + 5, LOW)])
def test_integers_are_not_cut_to_32_bits(seen, given, taken):
    binding.attn_decode(None, None, 1, 1, None, 1, None, 0, None, None, 1, given, 1.0, None, 0,
                        stream=0)
    assert seen["attn_decode"][11] == taken
    binding.attn_rope(None, None, None, None, 1, 1, 1, 1, 1, 64, 0, 0, 0, 0, None, pos0=given,
                      stream=0)
    assert seen["attn_rope"][16] == taken
    binding.attn_fwd_window(*[None] * 5, 1, 1, 1, 1, 64, 64, False, given, given, 1.0, stream=0)
    assert seen["attn_fwd_window"][12:14] == (taken, taken)
    binding.attn_fwd_ex(*[None] * 5, 1, 1, 1, 1, 64, 64, False, given, given, None, 1, 1, 1.0,
                        stream=0)
    assert seen["attn_fwd_ex"][12:14] == (taken, taken)
    binding.attn_bwd_window(*[None] * 9, 1, 1, 1, 1, 64, 64, False, given, given, 1.0, stream=0)
    assert seen["attn_bwd_window"][16:18] == (taken, taken)
    binding.attn_bwd_ex(*[None] * 9, 1, 1, 1, 1, 64, 64, False, given, given, None, 1, 1, 1.0,
                        stream=0)
    assert seen["attn_bwd_ex"][16:18] == (taken, taken)


def test_sizes_of_a_cache_beyond_32_bits_are_refused():
    one = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="2\\^31"):
        binding.PagedCache(one.expand(2 ** 32 + 3, 1, 1, 64), one.expand(2 ** 32 + 3, 1, 1, 64))


A = 0x10000  # an aligned, never-dereferenced stand-in address


@pytest.mark.parametrize("q,k,tq,tk,code", [
    (A, A, 0, 4, binding.ATTN_ERR_INVALID_ARG), (A, A, 4, 0, binding.ATTN_ERR_INVALID_ARG),
    (A, None, 4, -1, binding.ATTN_ERR_INVALID_ARG), (None, A, -1, 4, binding.ATTN_ERR_INVALID_ARG),
    (A, None, 0, 0, binding.ATTN_ERR_INVALID_ARG),
    (A, None, 2 ** 31 - 1, 0, binding.ATTN_ERR_UNSUPPORTED)])
def test_rotation_of_one_side_beside_none(q, k, tq, tk, code):
    """Only the side that is not given may have no rows."""
    rot = binding._RotationStruct(A, 0, 64, 0)
    assert binding.attn_rope(q, k, q, k, 1, 2, 2, tq, tk, 64, 0, 0, 0, 0, rot, stream=0,
                             pos0=1 if code == binding.ATTN_ERR_UNSUPPORTED else 0) == code
