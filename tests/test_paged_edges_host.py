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


def _append(**kw):
    a = dict(k=A, v=A, k_scale=None, v_scale=None, k_page_stride=16 * 4 * 64,
             k_token_stride=4 * 64, k_head_stride=64, v_page_stride=16 * 4 * 64,
             v_token_stride=4 * 64, v_head_stride=64, type=0, num_pages=10, page_size=16, heads=4,
             dqk=64, dv=64)
    a.update(kw)
    # (no new tokens: nothing is launched)
    return binding.attn_cache_append(binding._CacheStruct(**a), A, 4, 4, A, 2, 0, None, A, 0, A, 0,
                                     None, 0, None, 0, 0, stream=0)


@pytest.mark.parametrize("kw,ok", [
    (dict(), True),
    (dict(k_token_stride=64, k_head_stride=16 * 64), True),              # head-major pages
    (dict(k_page_stride=64, k_token_stride=640, k_head_stride=10240), True),  # pages innermost
    (dict(num_pages=1, k_page_stride=0, v_page_stride=0), True),
    (dict(page_size=1, k_token_stride=0, v_token_stride=0), True),
    (dict(heads=1, k_head_stride=0, v_head_stride=0), True),
    (dict(v_page_stride=2 ** 34, num_pages=2 ** 31 - 1), True),
    (dict(k_page_stride=0), False), (dict(v_page_stride=0), False),
    (dict(k_token_stride=0), False), (dict(v_head_stride=0), False),
    (dict(k_head_stride=56), False),                  # heads of 64 columns 56 apart
    (dict(k_token_stride=3 * 64), False),             # tokens inside their neighbours' heads
    (dict(v_page_stride=15 * 4 * 64), False),         # pages that share a token
    (dict(k_token_stride=64, k_head_stride=64), False),
    (dict(type=1, k_head_stride=48), False)])
def test_append_wants_rows_with_their_own_memory(kw, ok):
    assert _append(**kw) == (binding.ATTN_OK if ok else binding.ATTN_ERR_INVALID_ARG)


def test_a_broadcast_cache_is_not_appended_to():
    full = torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    new = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    for shared in (full[:1].expand(6, 16, 2, 64), full[:, :1].expand(6, 16, 2, 64),
                   full[:, :, :1].expand(6, 16, 2, 64),
                   full.flatten().as_strided((6, 16, 2, 64), (1024, 128, 64, 1))):
        for cache in (binding.PagedCache(shared, full), binding.PagedCache(full, shared)):
            with pytest.raises(ValueError, match="own memory"):
                binding.cache_append(cache, new, new, table, lens)
    big = torch.zeros(6, 3, 32, 4, 64, dtype=torch.bfloat16)
    for own in (full, full[::2, ::3, 1:], big[:, 1], big[:, 0, ::2, :, :].transpose(1, 2),
                big.permute(2, 0, 1, 3, 4)[:, :, 0], full[:1].expand(1, 16, 2, 64)):
        assert binding.PagedCache(own, own).rows_apart
