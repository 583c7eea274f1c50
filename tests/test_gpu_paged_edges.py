"""The rotation's, the cache's and the decode's helpers at the edges of what they take: integers
beyond 32 bits, sizes of zero, torch's modes, and the device status."""
import threading

import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import inv_freq, make_cache, make_table, rotate64, rotation_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from attention_backward_flashattention_gb300 import build
    build.build()
    binding.attn_cache_status()


def _rand(seed, *shape):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def _serving(lens=(100, 7, 300), page=16, heads=2, group=4, d=64):
    table, pages = make_table(list(lens), page, 3)
    cache = binding.PagedCache(make_cache(pages, page, heads, d, "bf16", "token", 4),
                               make_cache(pages, page, heads, d, "bf16", "token", 5))
    q = _rand(6, len(lens), heads * group, d)
    return cache, q, table, torch.tensor(lens, dtype=torch.int32).cuda()


# ---- integers beyond 32 bits --------------------------------------------------
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 70])
def test_windows_longer_than_any_sequence(window):
    cache, q, table, lens = _serving()
    want = binding.decode(cache, q, table, lens)
    got = binding.decode(cache, q, table, lens, window_left=window)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x = _rand(7, 1, 200, 2, 64)
    a = binding.forward(x, x, x, window=(window, 0))
    b = binding.forward(x, x, x, window=(200, 0))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = binding.backward(x, x, x, a[0], x, a[1], window=(window, 0), deterministic=True)
    gb = binding.backward(x, x, x, b[0], x, b[1], window=(200, 0), deterministic=True)
    assert all(torch.equal(s, t) for s, t in zip(ga, gb))


@pytest.mark.parametrize("window", [-2, -2 ** 31 - 1, -2 ** 32, -2 ** 32 + 5])
def test_negative_windows_are_refused(window):
    cache, q, table, lens = _serving()
    with pytest.raises(binding.AttnError):
        binding.decode(cache, q, table, lens, window_left=window)


@pytest.mark.parametrize("pos0", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -1, -2 ** 32 + 5])
def test_positions_beyond_32_bits_are_refused(pos0):
    x = _rand(8, 1, 4, 2, 64)
    with pytest.raises(binding.AttnError):
        binding.rope(x, x, binding.Rotation(inv_freq(64)), pos0=pos0)


@pytest.mark.parametrize("begin", [2 ** 32, 2 ** 32 + 16, -2 ** 32])
def test_columns_beyond_32_bits_are_refused(begin):
    x = _rand(8, 1, 4, 2, 64)
    with pytest.raises(binding.AttnError):
        binding.rope(x, x, binding.Rotation(inv_freq(32), begin=begin))


# ---- sizes of zero --------------------------------------------------------------
@pytest.mark.parametrize("width", [0, 4])
@pytest.mark.parametrize("given", [False, True])
def test_decode_of_an_empty_batch(width, given):
    cache, q, _, _ = _serving()
    table = torch.zeros(0, width, dtype=torch.int32, device="cuda")
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    out = (torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda"),
           torch.empty(0, 8, device="cuda")) if given else None
    o, lse = binding.decode(cache, q[:0], table, lens, out=out)
    assert o.shape == (0, 8, 64) and o.dtype == torch.bfloat16 and o.is_cuda
    assert lse.shape == (0, 8) and lse.dtype == torch.float32
    if given:
        assert o is out[0] and lse is out[1]
    else:
        assert binding.decode(cache, q[:0], table, lens, with_lse=False)[1] is None
    new = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert binding.cache_append(cache, new, new, table, lens, q=q[:0]).shape == (0, 8, 64)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("varlen", [False, True])
def test_queries_beside_no_keys(varlen, given):
    """Keys of no rows: the queries still turn, all of them in front of the first key."""
    q, k, freq = _rand(9, 1, 7, 2, 64), _rand(10, 1, 0, 3, 64), inv_freq(64)
    pos, kw = torch.arange(7) - 7 + 20, dict(pos0=20)
    if varlen:
        q, k = q[0], k[0]
        kw.update(cu_seqlens=[0, 3, 7], cu_seqlens_k=[0, 0, 0])
        pos = torch.tensor([-3, -2, -1, -4, -3, -2, -1]) + 20
    if given:
        kw["out"] = (torch.full_like(q, 7.0), torch.empty_like(k))
    rot = binding.Rotation(freq)
    qo, ko = binding.rope(q, k, rot, **kw)
    assert ko.shape == k.shape
    want, mag = rotate64(q.reshape(7, 2, 64), pos.cuda(), freq, 0, False)
    assert ((qo.reshape(7, 2, 64).double() - want).abs() <= rotation_bound(want, mag)).all()
    if given:
        assert qo is kw["out"][0]
    empty = binding.rope(q[..., :0, :, :], k, rot, pos0=20) if not varlen else \
        binding.rope(q[:0], k, rot, cu_seqlens=[0, 0], cu_seqlens_k=[0, 0])
    assert empty[0].numel() == 0 and empty[1].numel() == 0


# ---- torch's modes ----------------------------------------------------------------
def test_outputs_are_seen_by_dispatch_modes_and_deterministic_filling():
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.calls = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.calls.append(str(func))
            return func(*args, **(kwargs or {}))

    with Seen() as seen:
        binding._empty((3, 5), torch.bfloat16, torch.device("cuda", 0))
    assert any("empty" in c for c in seen.calls)
    was = torch.are_deterministic_algorithms_enabled()
    try:
        torch.use_deterministic_algorithms(True)
        x = binding._empty((3, 5), torch.bfloat16, torch.device("cuda", 0))
        assert torch.isnan(x).all()  # as torch.empty fills new memory there
    finally:
        torch.use_deterministic_algorithms(was)
    x = binding._empty((3, 5), torch.float32, torch.device("cuda", 0))
    assert x.shape == (3, 5) and x.is_contiguous()


def test_another_meaning_of_the_private_allocation_is_not_used(monkeypatch):
    device = torch.device("cuda", torch.cuda.current_device())
    for other in (lambda *a: torch.zeros(2, 3),
                  lambda *a: torch.empty(3, 2, device=device).t(),
                  lambda a, b: None):
        monkeypatch.setattr(binding, "_empty_strided", other)
        monkeypatch.setattr(binding, "_empty_is_known", False)
        x = binding._empty((4, 6), torch.bfloat16, device)
        assert x.shape == (4, 6) and x.is_contiguous() and x.is_cuda
        assert x.dtype == torch.bfloat16 and binding._empty_strided is None


# ---- the device status ------------------------------------------------------------
def test_no_error_is_lost_between_reading_and_clearing_the_status():
    """A call on another stream reports a bad page while the status is read all the time:
    every such report is read once the call is done."""
    cache, q, table, lens = _serving(lens=(5,))
    bad = table.clone()
    bad[:] = -1
    ws = binding.decode_workspace()
    out = binding.decode(cache, q, bad, lens, workspace=ws)
    torch.cuda.synchronize()
    assert binding.attn_cache_status() == binding.ATTN_ERR_BAD_PAGE
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    rounds, index = 300, torch.cuda.current_device()
    done, go = threading.Event(), threading.Event()
    failed = []

    def worker():
        try:
            torch.cuda.set_device(index)
            for _ in range(rounds):
                if not go.wait(60):
                    raise RuntimeError("not started")
                go.clear()
                binding.decode(cache, q, bad, lens, workspace=ws, out=out, stream=a)
                a.synchronize()
                done.set()
        except Exception as e:  # (for the reader to see)
            failed.append(e)
            done.set()

    t = threading.Thread(target=worker)
    t.start()
    lost = 0
    for _ in range(rounds):
        done.clear()
        go.set()
        found = 0
        while not done.is_set():
            found += binding.attn_cache_status(b) == binding.ATTN_ERR_BAD_PAGE
        found += binding.attn_cache_status(b) == binding.ATTN_ERR_BAD_PAGE
        lost += found == 0
        if failed:
            break
    t.join(60)
    assert not failed, failed
    assert lost == 0 and binding.attn_cache_status() == binding.ATTN_OK


def test_status_read_on_many_threads():
    """Each report is read by one of the readers, by one alone."""
    cache, q, table, lens = _serving(lens=(5,))
    bad = table.clone()
    bad[:] = -1
    ws = binding.decode_workspace()
    index = torch.cuda.current_device()
    for _ in range(20):
        binding.decode(cache, q, bad, lens, workspace=ws)
        torch.cuda.synchronize()
        got = []

        def read():
            torch.cuda.set_device(index)
            s = torch.cuda.Stream()
            got.append(binding.attn_cache_status(s))

        readers = [threading.Thread(target=read) for _ in range(8)]
        for r in readers:
            r.start()
        for r in readers:
            r.join(60)
        assert sorted(got) == [binding.ATTN_ERR_BAD_PAGE] + [binding.ATTN_OK] * 7
