"""Rotation, paged cache and decode: what is decided on the host (no GPU needed) —
refusals of the C entry points and of the Python helpers, the fixed-point rates and
the workspace's size."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from attention_backward_flashattention_gb300 import build as build_mod

A = 0x10000  # an aligned, never-dereferenced stand-in address


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return binding.load()


def _rot(**kw):
    a = dict(rates=A, begin=0, dim=64, style=0)
    a.update(kw)
    return binding._RotationStruct(**a)


def _cache(**kw):
    a = dict(k=A, v=A, k_scale=None, v_scale=None, k_page_stride=64 * 4 * 64,
             k_token_stride=4 * 64, k_head_stride=64, v_page_stride=64 * 4 * 64,
             v_token_stride=4 * 64, v_head_stride=64, type=0, num_pages=10, page_size=64, heads=4,
             dqk=64, dv=64)
    a.update(kw)
    return binding._CacheStruct(**a)


def _rope(**kw):
    a = dict(q=A, k=A, q_out=A, k_out=A, B=2, Hq=4, Hk=2, Tq=16, Tk=16, d=64, q_row=0, k_row=0,
             q_out_row=0, k_out_row=0, rotation=_rot(), inverse=0, pos0=0, cu_seqlens_q=None,
             cu_seqlens_k=None, stream=0)
    a.update(kw)
    return binding.attn_rope(**a)


def _append(**kw):
    a = dict(cache=_cache(), block_table=A, max_pages=4, table_stride=4, lens=A, B=2, T=6,
             cu_seqlens=None, k=A, k_row=0, v=A, v_row=0, q=A, q_row=0, q_out=A, q_out_row=0,
             Hq=8, rotation=_rot(), stream=0)
    a.update(kw)
    return binding.attn_cache_append(**a)


def _decode(**kw):
    a = dict(cache=_cache(), block_table=A, max_pages=4, table_stride=4, lens=A, B=2, q=A, q_row=0,
             o=A, lse=A, Hq=8, window_left=-1, scale=0.125, workspace=A,
             workspace_bytes=binding.attn_decode_workspace_size(), stream=0)
    a.update(kw)
    return binding.attn_decode(**a)


INV, UNS = binding.ATTN_ERR_INVALID_ARG, binding.ATTN_ERR_UNSUPPORTED

BAD_ROTATIONS = [dict(rates=None), dict(rates=A + 4), dict(begin=8), dict(begin=-16), dict(dim=0),
                 dict(dim=24), dict(dim=-16), dict(dim=80), dict(begin=16, dim=64),
                 dict(begin=80, dim=16), dict(begin=2147483632, dim=16), dict(style=2)]


@pytest.mark.parametrize("kw,code", [
    (dict(q=None, k=None, q_out=None, k_out=None), INV), (dict(q=None), INV),
    (dict(q_out=None), INV), (dict(k_out=None), INV), (dict(rotation=None), INV),
    (dict(q=A + 8), INV), (dict(k_out=A + 2), INV), (dict(B=0), INV), (dict(Tq=0), INV),
    (dict(Tk=-1), INV), (dict(Hq=0), INV), (dict(Hk=0), INV), (dict(pos0=-1), INV),
    (dict(d=96), UNS), (dict(d=256), UNS), (dict(q_row=255), INV), (dict(q_row=252), INV),
    (dict(k_row=64), INV), (dict(q_out_row=-256), INV),
    (dict(pos0=2147483640), UNS), (dict(B=1 << 20, Tq=1 << 12), UNS),
    (dict(Hq=1 << 20), UNS),
    (dict(cu_seqlens_k=[0, 8, 16]), INV),
    (dict(cu_seqlens_q=[0, 8, 15]), INV), (dict(cu_seqlens_q=[1, 8, 16]), INV),
    (dict(cu_seqlens_q=[0, 17, 16]), INV),
    (dict(cu_seqlens_q=[0, 8, 16], cu_seqlens_k=[0, 8, 17]), INV),
    (dict(B=1025, Tq=1025, Tk=1025, cu_seqlens_q=list(range(1026))), UNS),
] + [(dict(rotation=_rot(**r)), INV) for r in BAD_ROTATIONS])
def test_rope_rejects(kw, code):
    assert _rope(**kw) == code


BAD_CACHES = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(k=A + 8), INV), (dict(type=2), INV),
    (dict(num_pages=0), INV), (dict(page_size=0), INV), (dict(heads=0), INV),
    (dict(page_size=-1), INV), (dict(dqk=96, dv=96), UNS), (dict(dqk=128, dv=64), UNS),
    (dict(dqk=64, dv=128), UNS), (dict(k_token_stride=4), INV), (dict(k_page_stride=-8), INV),
    (dict(v_head_stride=65), INV), (dict(k_scale=A), INV),  # scales are for e4m3
    (dict(type=1, k_head_stride=72), INV),                  # 8-bit rows: multiples of 16
    (dict(type=1, v_scale=A + 2), INV),
]
BAD_TABLES = [
    (dict(cache=None), INV), (dict(block_table=None), INV), (dict(lens=None), INV),
    (dict(block_table=A + 2), INV), (dict(lens=A + 1), INV), (dict(B=0), INV),
    (dict(max_pages=0), INV), (dict(table_stride=3), INV),
] + [(dict(cache=_cache(**c)), code) for c, code in BAD_CACHES]


@pytest.mark.parametrize("kw,code", BAD_TABLES + [
    (dict(k=None), INV), (dict(v=None), INV), (dict(q=None), INV), (dict(q_out=None), INV),
    (dict(k=A + 8), INV), (dict(q_out=A + 8), INV), (dict(Hq=0), INV), (dict(T=-2), INV),
    (dict(T=5), INV),                                       # not a multiple of B
    (dict(k_row=128), INV), (dict(v_row=260), INV), (dict(q_row=8), INV),
    (dict(cu_seqlens=[0, 3, 5]), INV), (dict(cu_seqlens=[0, 7, 6]), INV),
    (dict(B=1025, T=1025, cu_seqlens=list(range(1026))), UNS),
] + [(dict(rotation=_rot(**r)), INV) for r in BAD_ROTATIONS])
def test_append_rejects(kw, code):
    assert _append(**kw) == code


def test_append_of_nothing_launches_nothing():
    assert _append(T=0, q=None, q_out=None) == binding.ATTN_OK


@pytest.mark.parametrize("scale", [1e-45, 1e-39, 3e38])
def test_decode_rejects_scales_whose_factor_is_no_normal_number(scale):
    assert _decode(scale=scale) == INV


@pytest.mark.parametrize("kw,code", BAD_TABLES + [
    (dict(q=None), INV), (dict(o=None), INV), (dict(q=A + 8), INV), (dict(o=A + 8), INV),
    (dict(lse=A + 2), INV), (dict(Hq=0), INV), (dict(Hq=6), INV), (dict(q_row=128), INV),
    (dict(window_left=-2), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(workspace=None), INV),
    (dict(workspace=A + 128), INV), (dict(B=(1 << 20) + 1), UNS), (dict(Hq=1 << 16), UNS),
    (dict(workspace_bytes=binding.ATTN_OK), binding.ATTN_ERR_WORKSPACE_TOO_SMALL),
])
def test_decode_rejects(kw, code):
    assert _decode(**kw) == code


def test_workspace():
    n = binding.attn_decode_workspace_size()
    assert n % 256 == 0
    # header, counters, and two partial results of 32 rows for each of 3 * 304 pieces
    slots = 2 * 3 * 304
    assert n == 256 + -(-4 * slots * 4 // 256) * 256 + slots * 32 * (2 + 128) * 4
    assert binding.attn_decode_workspace_init(None, n, 0) == INV
    assert binding.attn_decode_workspace_init(A + 16, n, 0) == INV
    assert binding.attn_decode_workspace_init(A, n - 1, 0) == binding.ATTN_ERR_WORKSPACE_TOO_SMALL


def test_error_texts():
    assert "page" in binding.attn_strerror(binding.ATTN_ERR_BAD_PAGE)
    assert "initialised" in binding.attn_strerror(binding.ATTN_ERR_WORKSPACE_NOT_READY)


# pi to 60 digits
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


@pytest.mark.parametrize("rate", [1.0, 0.1, 0.75, 1e-4, 1e-12, 2.0 * math.pi, math.pi, 123.456,
                                  1e5, -1.0, -0.3, 0.0])
def test_rates_are_turns(rate):
    """Within a few units of 2^-64 of a turn (a whole turn up or down is the same angle)."""
    word = binding.attn_rope_rates([rate])[0]
    turn = Fraction(rate) / (2 * PI)
    exact = (turn - math.floor(turn)) * 2 ** 64
    off = abs(word - exact)
    off = min(off, 2 ** 64 - off)
    # the product is exact to 2^-105 of its size and each half is cut to a unit
    assert off <= 2 + abs(turn) * Fraction(1, 2 ** 40), float(off)


def test_rates_reject():
    for bad in ([math.nan], [1.0, math.inf], []):
        with pytest.raises(binding.AttnError):
            binding.attn_rope_rates(bad)
    out = (ctypes.c_ulonglong * 1)()
    src = (ctypes.c_double * 1)(1.0)
    f = binding.load().attn_rope_rates
    assert f(None, 1, ctypes.cast(out, ctypes.c_void_p)) == INV
    assert f(ctypes.cast(src, ctypes.c_void_p), 1, None) == INV


# ---- Python helpers (CPU tensors: refused or checked before any launch) ----
def test_rotation_object():
    r = binding.Rotation([1.0, 0.5] * 8, begin=16, interleaved=True, device="cpu")
    assert (r.dim, r.begin, r.struct.style) == (32, 16, binding.ROPE_PAIRS)
    words = [w % (1 << 64) for w in r.rates.tolist()]
    assert words == binding.attn_rope_rates([1.0, 0.5] * 8)


def _tensors(kind=torch.bfloat16, d=64):
    return torch.zeros(3, 16, 2, d, dtype=kind), torch.zeros(3, 16, 2, d, dtype=kind)


def test_paged_cache_describes_strides():
    k, v = _tensors()
    s = binding.PagedCache(k.transpose(1, 2).contiguous().transpose(1, 2), v).struct
    assert (s.k_page_stride, s.k_token_stride, s.k_head_stride) == (2048, 64, 1024)
    assert (s.v_page_stride, s.v_token_stride, s.v_head_stride) == (2048, 128, 64)
    assert (s.num_pages, s.page_size, s.heads, s.dqk, s.dv, s.type) == (3, 16, 2, 64, 64, 0)


def test_paged_cache_rejects():
    k, v = _tensors()
    for bad in ((k[0], v[0]), (k, v[:2]), (k.float(), v.float()), (k, v.to(torch.float8_e4m3fn)),
                (k.transpose(2, 3), v.transpose(2, 3)), (k, v, torch.ones(3)),
                (k, v, torch.ones(2).double())):
        with pytest.raises(ValueError):
            binding.PagedCache(*bad)


def test_rows_of_views():
    rows = lambda t: binding._rows(t, t.shape, "x")
    x = torch.zeros(2, 5, 3, 4, 64, dtype=torch.bfloat16)
    assert rows(x.select(2, 1)) == 3 * 4 * 64                 # a slot of a packed buffer
    assert rows(torch.zeros(7, 4, 64, dtype=torch.bfloat16)) == 256
    assert rows(x[:, :1, 0]) == 5 * 3 * 4 * 64                # one row per batch
    with pytest.raises(ValueError, match="evenly"):
        rows(x[:, :4, 0])
    with pytest.raises(ValueError, match="adjacent"):
        rows(x[:, :, 0].transpose(1, 2))
    with pytest.raises(ValueError, match="bfloat16"):
        rows(x[:, :, 0].float())
    one = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    assert rows(one[:, :2]) == 128                            # a single row: any distance does
    for broadcast in (one.expand(5, 4, 64), one[None].expand(3, 1, 4, 64),
                      x[:1, :, 0].expand(2, 5, 4, 64), x[:, :1, 0].expand(2, 5, 4, 64)):
        with pytest.raises(ValueError, match="evenly|own memory"):
            rows(broadcast)


def test_tables_of_views():
    cache = binding.PagedCache(*_tensors())
    lens = torch.zeros(3, dtype=torch.int32)
    big = torch.zeros(3, 10, dtype=torch.int32)
    assert binding._check_tables(cache, big, lens) == (3, 10, 10)
    assert binding._check_tables(cache, big[:, 2:6], lens) == (3, 4, 10)
    assert binding._check_tables(cache, big[:1, 2:6], lens[:1]) == (1, 4, 4)
    for bad in (big[:1].expand(3, 10), big[:, :1].expand(3, 10), big[:, ::2], big.t()[:3]):
        with pytest.raises(ValueError):
            binding._check_tables(cache, bad, lens)


def _refused(call, *args, **kw):
    with pytest.raises(ValueError) as e:
        call(*args, **kw)
    return str(e.value)


def test_helpers_reject_shapes():
    k, v = _tensors()
    cache = binding.PagedCache(k, v)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    new = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    rot = binding.Rotation([1.0] * 32, device="cpu")
    for a in (dict(block_table=table.long()), dict(lens=lens.long()), dict(lens=lens[:1]),
              dict(k=new[:1]), dict(k=new.float()), dict(v=new[:, :1]), dict(q=q[:1]),
              dict(q=None, q_out=q), dict(cu_seqlens=[0, 2]), dict(q=q[:, :, :32])):
        args = dict(k=new, v=new, block_table=table, lens=lens, q=q)
        args.update(a)
        assert "CUDA" not in _refused(binding.cache_append, cache, **args), a
    for a in (dict(q=q[:1]), dict(q=q.float()), dict(lens=lens.float()),
              dict(out=(torch.zeros(2, 4, 64), None)), dict(out=(q, torch.zeros(2, 3)))):
        args = dict(q=q, block_table=table, lens=lens, workspace=torch.zeros(8, dtype=torch.uint8))
        args.update(a)
        assert "CUDA" not in _refused(binding.decode, cache, **args), a
    x = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16)
    for a in ((None, None, rot), (x, x[:1], rot), (x[0], x[0], rot), (x.float(), x, rot),
              (x, x[..., :32], rot)):
        assert "CUDA" not in _refused(binding.rope, *a)
    assert "CUDA" not in _refused(binding.rope, x, x, rot, out=(x, None))


def test_offsets_of_another_length_are_not_read_past_their_end():
    x = torch.zeros(16, 4, 64, dtype=torch.bfloat16)
    rot = binding.Rotation([1.0] * 32, device="cpu")
    for cu_k in ([0, 16], [0, 4, 8, 16], []):
        assert "same length" in _refused(binding.rope, x, x, rot, cu_seqlens=[0, 8, 16],
                                         cu_seqlens_k=cu_k)


def test_a_broadcast_workspace_is_no_workspace():
    cache = binding.PagedCache(*_tensors())
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    ws = torch.zeros(1, dtype=torch.uint8).expand(binding.attn_decode_workspace_size())
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    assert "workspace" in _refused(binding.decode, cache, q, table, lens, workspace=ws)


def test_helpers_reject_host_tensors():
    """A host pointer never reaches a kernel."""
    k, v = _tensors()
    cache = binding.PagedCache(k, v)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    new = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    rot = binding.Rotation([1.0] * 32, device="cpu")
    assert "CUDA" in _refused(binding.cache_append, cache, new, new, table, lens)
    assert "CUDA" in _refused(binding.decode, cache, new, table, lens)
    x = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16)
    assert "CUDA" in _refused(binding.rope, x, x, rot)
