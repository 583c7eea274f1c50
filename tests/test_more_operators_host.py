"""Grouped heads, prefill and head norms: what is decided on the host (no GPU needed) — refusals
of the C entry points and of the Python helpers, and sizes of workspaces."""
import ctypes

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from attention_backward_flashattention_gb300 import build as build_mod
from tests.test_paged_host import A, BAD_ROTATIONS, BAD_TABLES, INV, UNS, _cache, _rot

SMALL = binding.ATTN_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return binding.load()


# ---------------------------------------------------------------------------- grouped heads
def _rows(**kw):
    return binding._RowsStruct(**kw)


def _fwd(**kw):
    a = dict(q=A, k=A, v=A, o=A, lse=A, B=2, Hq=8, Hk=2, Tq=128, Tk=128, dqk=64, dv=64, rows=None,
             causal=1, window_left=-1, window_right=-1, scale=0.125, cu_seqlens_q=None,
             cu_seqlens_k=None, stream=0)
    a.update(kw)
    return binding.attn_fwd_grouped(**a)


def _bwd(**kw):
    a = dict(q=A, k=A, v=A, o=A, dO=A, lse=A, dq=A, dk=A, dv_out=A, B=2, Hq=8, Hk=2, Tq=128,
             Tk=128, dqk=64, dv=64, rows=None, causal=1, window_left=-1, window_right=-1,
             scale=0.125, cu_seqlens_q=None, cu_seqlens_k=None, deterministic=0, workspace=A,
             workspace_bytes=1 << 40, stream=0)
    a.update(kw)
    return binding.attn_bwd_grouped(**a)


GROUPED = [
    (dict(q=None), INV), (dict(k=A + 8), INV), (dict(o=None), INV), (dict(Hk=0), INV),
    (dict(Hk=3), INV), (dict(Hq=0), INV), (dict(Hq=-8), INV), (dict(Hk=-2), INV), (dict(B=0), INV),
    (dict(Tq=0), INV), (dict(Tk=0), INV), (dict(dqk=96, dv=96), UNS), (dict(dqk=128, dv=64), UNS),
    (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(Tq=129), UNS),  # causal with more queries than keys
    (dict(causal=0, window_left=4, Tq=129), UNS), (dict(window_left=-2), INV),
    (dict(Hq=1 << 14, Hk=1), UNS),
    (dict(rows=_rows(q=504)), INV), (dict(rows=_rows(k=64)), INV), (dict(rows=_rows(v=132)), INV),
    (dict(rows=_rows(o=-512)), INV), (dict(rows=_rows(q=1 << 40)), INV),
    (dict(cu_seqlens_k=[0, 64, 128]), INV), (dict(cu_seqlens_q=[0, 64, 127]), INV),
    (dict(cu_seqlens_q=[0, 130, 128]), INV),
    (dict(cu_seqlens_q=[0, 64, 128], cu_seqlens_k=[0, 60, 128]), UNS),
    (dict(cu_seqlens_q=[0, 64, 128], cu_seqlens_k=[0, 0, 128], causal=0), INV),
    (dict(B=1025, cu_seqlens_q=[0] * 1025 + [128]), UNS),
]


@pytest.mark.parametrize("kw,code", GROUPED + [(dict(lse=A + 2), INV)])
def test_forward_rejects(kw, code):
    assert _fwd(**kw) == code


@pytest.mark.parametrize("kw,code", GROUPED + [
    (dict(lse=None), INV), (dict(dO=A + 8), INV), (dict(dk=None), INV), (dict(workspace=None), INV),
    (dict(workspace=A + 128), INV), (dict(workspace_bytes=1000), SMALL),
    (dict(rows=_rows(dk=96)), INV), (dict(rows=_rows(d_o=508)), INV), (dict(rows=_rows(dq=8)), INV),
])
def test_backward_rejects(kw, code):
    assert _bwd(**kw) == code


def test_grouped_workspace():
    size, own = binding.attn_bwd_grouped_workspace_size, binding.attn_bwd_workspace_size
    # many key tiles and heads: the groups stay whole
    assert size(4, 32, 8, 2048, 2048, 128, 128) == own(4, 32, 2048, 2048, 128, 128)
    # as many key heads as query heads: nothing to split
    assert size(1, 4, 4, 128, 128, 64, 64) == own(1, 4, 128, 128, 64, 64)
    # few: fp32 sums of dK and dV, a part for each query head at most
    need = size(1, 16, 1, 128, 128, 128, 128)
    assert need == own(1, 16, 128, 128, 128, 128) + 128 * 16 * 256 * 4
    assert _bwd(B=1, Hq=16, Hk=1, Tq=128, Tk=128, dqk=128, dv=128,
                workspace_bytes=need - 1) == SMALL
    for bad in ((0, 8, 2, 8, 8, 64, 64), (1, 8, 3, 8, 8, 64, 64), (1, 8, 2, 8, 8, 64, 128),
                (1, 8, 0, 8, 8, 64, 64), (1, 8, 2, 8, 0, 64, 64)):
        assert size(*bad) == 0


def test_helpers_reject_grouped():
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    q, k = t(1, 8, 4, 64), t(1, 8, 2, 64)
    with pytest.raises(ValueError, match="block mask"):
        binding.forward(q, k, k, block_mask=torch.ones(1, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="multiple"):
        binding.forward(q, t(1, 8, 3, 64), t(1, 8, 3, 64))
    with pytest.raises(ValueError, match="agree"):
        binding.forward(q, k, t(1, 8, 1, 64))
    with pytest.raises(ValueError, match="agree"):
        binding.forward(q, t(2, 8, 2, 64), t(2, 8, 2, 64))
    with pytest.raises(ValueError, match="head size"):
        binding.forward(q, t(1, 8, 2, 128), k)
    with pytest.raises(ValueError, match="CUDA"):
        binding.forward(q, k, k)
    with pytest.raises(ValueError, match="bfloat16"):
        binding.forward(q.float(), k, k)
    with pytest.raises(ValueError, match="own memory"):  # a broadcast tensor
        binding.forward(q, t(1, 1, 2, 64).expand(1, 8, 2, 64), k)
    with pytest.raises(ValueError, match="adjacent"):
        binding.forward(q, t(1, 2, 8, 64).transpose(1, 2), k)
    lse = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="o and dO"):
        binding.backward(q, k, k, q, t(1, 8, 2, 64), lse)
    with pytest.raises(ValueError, match="lse"):
        binding.backward(q, k, k, q, q, lse[..., :4])
    with pytest.raises(ValueError, match="out must"):
        binding.backward(q, k, k, q, q, lse, out=(q, q, k))
    with pytest.raises(ValueError, match="workspace"):
        binding.backward(q, k, k, q, q, lse, workspace=torch.zeros(64, 2)[:, 0])


# ---------------------------------------------------------------------------- prefill
def _prefill(**kw):
    a = dict(cache=_cache(), block_table=A, max_pages=4, table_stride=4, lens=A, B=2, T=6,
             cu_seqlens=None, q=A, q_row=0, o=A, lse=A, Hq=8, window_left=-1, scale=0.125,
             workspace=A, workspace_bytes=binding.attn_prefill_workspace_size(), stream=0)
    a.update(kw)
    return binding.attn_prefill(**a)


@pytest.mark.parametrize("kw,code", BAD_TABLES + [
    (dict(q=None), INV), (dict(q=A + 8), INV), (dict(o=None), INV), (dict(o=A + 8), INV),
    (dict(lse=A + 2), INV), (dict(workspace=None), INV), (dict(workspace=A + 16), INV),
    (dict(Hq=0), INV), (dict(Hq=6), INV), (dict(Hq=4 * 129), UNS), (dict(T=-2), INV),
    (dict(T=5), INV), (dict(window_left=-2), INV), (dict(q_row=8), INV), (dict(q_row=516), INV),
    (dict(q_row=1 << 40), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=1e-39), INV), (dict(scale=3e38), INV), (dict(scale=float("nan")), INV),
    (dict(cu_seqlens=[0, 3, 5]), INV), (dict(cu_seqlens=[0, 7, 6]), INV),
    (dict(cu_seqlens=[1, 3, 6]), INV),
    (dict(B=1025, T=1025, cu_seqlens=list(range(1026))), UNS),
    (dict(workspace_bytes=1000), SMALL),
])
def test_prefill_rejects(kw, code):
    assert _prefill(**kw) == code


def test_prefill_of_nothing_launches_nothing():
    assert _prefill(T=0) == binding.ATTN_OK
    assert _prefill(T=0, cu_seqlens=[0, 0, 0]) == binding.ATTN_OK


def test_helper_rejects_prefill():
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    cache = binding.PagedCache(t(4, 16, 2, 64), t(4, 16, 2, 64))
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ok = dict(cache=cache, q=t(6, 4, 64), block_table=table, lens=lens)
    call = lambda **kw: binding.prefill(**{**ok, **kw})
    for bad, what in ((dict(q=t(6, 4, 128)), "T, heads"), (dict(q=t(6, 256)), "T, heads"),
                      (dict(q=t(6, 4, 64).float()), "bfloat16"),
                      (dict(cu_seqlens=[0, 6]), "one entry more"),
                      (dict(lens=lens.long()), "lens"), (dict(block_table=table.long()), "int32"),
                      (dict(out=(t(6, 4, 128), None)), "out"),
                      (dict(out=(t(6, 4, 64), torch.zeros(4, 6))), "out"),
                      (dict(workspace=torch.zeros(64, 2)[:, 0]), "workspace"), ({}, "CUDA")):
        with pytest.raises(ValueError, match=what):
            call(**bad)
    with pytest.raises(ValueError, match="CUDA"):
        binding.prefill_workspace("cpu")


# ---------------------------------------------------------------------------- head norms
def _norm(**kw):
    a = dict(q_weight=A, k_weight=A, eps=1e-6)
    a.update(kw)
    return binding._NormStruct(**a)


def _norm_rope(**kw):
    a = dict(q=A, k=A, q_out=A, k_out=A, B=2, Hq=4, Hk=2, Tq=16, Tk=16, d=64, q_row=0, k_row=0,
             q_out_row=0, k_out_row=0, norm=_norm(), rotation=_rot(), pos0=0, cu_seqlens_q=None,
             cu_seqlens_k=None, stream=0)
    a.update(kw)
    return binding.attn_norm_rope(**a)


def _norm_bwd(**kw):
    a = dict(q=A, k=A, dq_out=A, dk_out=A, dq=A, dk=A, dq_weight=A, dk_weight=A, B=2, Hq=4, Hk=2,
             Tq=16, Tk=16, d=64, rows=None, norm=_norm(), rotation=_rot(), pos0=0,
             cu_seqlens_q=None, cu_seqlens_k=None, workspace=A, workspace_bytes=1 << 30, stream=0)
    a.update(kw)
    return binding.attn_norm_rope_bwd(**a)


BAD_NORMS = [dict(q_weight=A + 2), dict(k_weight=A + 1), dict(eps=0.0), dict(eps=-1e-6),
             dict(eps=1e-39), dict(eps=float("inf")), dict(eps=float("nan"))]
NORMS = [
    (dict(norm=None), INV), (dict(q=A + 8), INV), (dict(k=None), INV), (dict(B=0), INV),
    (dict(Tq=0), INV), (dict(Tk=-1), INV), (dict(Hq=0), INV), (dict(Hk=0), INV),
    (dict(pos0=-1), INV), (dict(d=96), UNS), (dict(pos0=2147483640), UNS),
    (dict(B=1 << 20, Tq=1 << 12), UNS), (dict(Hq=1 << 20), UNS),
    (dict(cu_seqlens_k=[0, 8, 16]), INV), (dict(cu_seqlens_q=[0, 8, 15]), INV),
    (dict(cu_seqlens_q=[0, 17, 16]), INV),
    (dict(cu_seqlens_q=[0, 8, 16], cu_seqlens_k=[0, 8, 17]), INV),
    (dict(B=1025, Tq=1025, Tk=1025, cu_seqlens_q=list(range(1026))), UNS),
] + [(dict(norm=_norm(**n)), INV) for n in BAD_NORMS] + \
    [(dict(rotation=_rot(**r)), INV) for r in BAD_ROTATIONS]


@pytest.mark.parametrize("kw,code", NORMS + [
    (dict(q=None, k=None, q_out=None, k_out=None), INV), (dict(q_out=None), INV),
    (dict(k_out=A + 2), INV), (dict(q_row=255), INV), (dict(k_row=64), INV),
    (dict(q_out_row=-256), INV),
])
def test_norm_rope_rejects(kw, code):
    assert _norm_rope(**kw) == code


def _norm_rows(**kw):
    return binding._NormRowsStruct(**kw)


@pytest.mark.parametrize("kw,code", NORMS + [
    (dict(dq_out=None), INV), (dict(dk=None), INV), (dict(q=None, dq_out=None, dq=None), INV),
    (dict(dq_out=A + 8), INV), (dict(dk_weight=A + 2), INV), (dict(workspace=None), INV),
    (dict(workspace=A + 64), INV), (dict(workspace_bytes=100), SMALL),
    (dict(rows=_norm_rows(q=255)), INV), (dict(rows=_norm_rows(dk_out=64)), INV),
    (dict(rows=_norm_rows(dq=8)), INV),
])
def test_norm_rope_backward_rejects(kw, code):
    assert _norm_bwd(**kw) == code


def test_norm_workspace():
    assert binding.attn_norm_rope_bwd_workspace_size(96) == 0
    assert binding.attn_norm_rope_bwd_workspace_size(192) == \
        3 * binding.attn_norm_rope_bwd_workspace_size(64)


@pytest.mark.parametrize("norm", BAD_NORMS)
def test_append_with_a_bad_norm(norm):
    assert binding.attn_cache_append_norm(
        _cache(), A, 4, 4, A, 2, 6, None, A, 0, A, 0, A, 0, A, 0, 8, norm=_norm(**norm),
        rotation=_rot(), stream=0) == INV


@pytest.mark.parametrize("kw,code", BAD_TABLES)
def test_append_with_a_norm_rejects(kw, code):
    a = dict(cache=_cache(), block_table=A, max_pages=4, table_stride=4, lens=A, B=2, T=6,
             cu_seqlens=None, k=A, k_row=0, v=A, v_row=0, q=A, q_row=0, q_out=A, q_out_row=0,
             Hq=8, norm=_norm(), rotation=_rot(), stream=0)
    a.update(kw)
    assert binding.attn_cache_append_norm(**a) == code


def test_helpers_reject_norms():
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="fp32"):
        binding.HeadNorm(t(64))
    with pytest.raises(ValueError, match="fp32"):
        binding.HeadNorm(torch.zeros(64, 2)[:, 0])
    norm = binding.HeadNorm(torch.ones(64), torch.ones(64))
    q, k = t(1, 8, 4, 64), t(1, 8, 2, 64)
    for args, kw, what in (((None, None), {}, "both None"), ((t(8, 4, 64), k), {}, "dimensions"),
                           ((q, t(2, 8, 2, 64)), {}, "agree"),
                           ((t(1, 8, 4, 128), None), {}, "one value per column"),
                           ((q, k), dict(out=(q, None)), "like k"),
                           ((q, k), dict(cu_seqlens_k=[0, 8]), "needs cu_seqlens"),
                           ((q, k), {}, "CUDA")):
        with pytest.raises(ValueError, match=what):
            binding.norm_rope(*args, norm, **kw)
    with pytest.raises(ValueError, match="like q"):
        binding.norm_rope_backward(q, k, k, k, norm)
    with pytest.raises(ValueError, match="workspace"):
        binding.norm_rope_backward(q, k, q, k, norm, workspace=torch.zeros(64, 2)[:, 0])
    cache = binding.PagedCache(t(4, 16, 2, 64), t(4, 16, 2, 64))
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.cache_append(cache, t(2, 2, 64), t(2, 2, 64), table, lens, norm=norm)


def test_structures_match_the_header():
    assert ctypes.sizeof(binding._RowsStruct) == 8 * 8
    assert ctypes.sizeof(binding._NormStruct) == 24
    assert ctypes.sizeof(binding._NormRowsStruct) == 6 * 8
