"""attn_cache_append on the GPU against the plain form: layouts, both cache types, ragged and
unused rows, page ends, far positions, bad pages, and what must stay as it was."""
import pytest
import torch

from attention_backward_flashattention_gb300 import binding
from tests.paged_common import (E4M3_HALF, bits, inv_freq, make_cache, make_table, rotate64,
                                rotation_bound)

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


class Case:
    def __init__(self, d, kind, order, page, past, new, hq=4, heads=2, begin=0, dim=0, inter=False,
                 scales=True, seed=1, extra_len=None):
        dqk, dv = d
        self.kind, self.page, self.new = kind, page, new
        self.lens = [p + n for p, n in zip(past, new)]
        self.table, pages = make_table(self.lens, page, seed)
        self.kc = make_cache(pages, page, heads, dqk, kind, order, seed + 1)
        self.vc = make_cache(pages, page, heads, dv, kind, order, seed + 2)
        g = torch.Generator(device="cpu").manual_seed(seed + 3)
        e = kind == "e4m3" and scales
        self.ks = (torch.rand(heads, generator=g) / 40 + 0.01).cuda() if e else None
        self.vs = (torch.rand(heads, generator=g) / 40 + 0.01).cuda() if e else None
        T = sum(new)
        row = _rand(seed + 4, T, hq * dqk + heads * (dqk + dv))  # slices of one projection
        q, k, v = row.split([hq * dqk, heads * dqk, heads * dv], 1)
        self.q, self.k, self.v = (q.unflatten(1, (hq, dqk)), k.unflatten(1, (heads, dqk)),
                                  v.unflatten(1, (heads, dv)))
        self.freq, self.begin, self.inter = inv_freq(dim) if dim else [], begin, inter
        self.rot = binding.Rotation(self.freq, begin=begin, interleaved=inter) if dim else None
        self.pos = torch.cat([torch.arange(n) + p for p, n in zip(past, new)]).cuda()
        self.seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
        self.cu = None if len(set(new)) == 1 else [sum(new[:i]) for i in range(len(new) + 1)]
        self.cache = binding.PagedCache(self.kc, self.vc, self.ks, self.vs)
        self.before = (self.kc.clone(), self.vc.clone())

    def lens_t(self):
        return torch.tensor(self.lens, dtype=torch.int32).cuda()

    def append(self, **kw):
        return binding.cache_append(self.cache, self.k, self.v, self.table, self.lens_t(),
                                    q=self.q, rotation=self.rot, cu_seqlens=self.cu, **kw)

    def turned(self, x):
        if not self.freq:
            return x.double(), torch.zeros(x.shape, dtype=torch.float64).cuda()
        return rotate64(x, self.pos, self.freq, self.begin, self.inter)

    def check(self, q_out, written=None):
        """written: mask over tokens that reach the cache (None: all)."""
        want, mag = self.turned(self.q)
        assert ((q_out.double() - want).abs() <= rotation_bound(want, mag)).all()
        w = torch.ones(len(self.pos), dtype=torch.bool).cuda() if written is None else written
        slots = self.table.long()[self.seq[w], self.pos[w] // self.page]
        at = (slots, self.pos[w] % self.page)
        for cache, before, x, scale, turn in ((self.kc, self.before[0], self.k, self.ks, True),
                                              (self.vc, self.before[1], self.v, self.vs, False)):
            got = bits(cache)[at].view(cache.dtype).double()
            want, mag = self.turned(x) if turn else (x.double(), torch.zeros_like(x).double())
            want, mag = want[w], mag[w]
            if self.kind == "bf16":
                bound = rotation_bound(want, mag)
                if not turn:
                    bound = torch.zeros_like(bound)
            else:
                unit = 1.0 if scale is None else scale.double()[:, None]
                want, mag = (want / unit).clamp(-448, 448), mag / unit
                # half a step of e4m3 (2^-10 below 2^-6), fp32 arithmetic before it
                err = 2.0 ** -20 * mag + 2.0 ** -24 * want.abs()
                bound = torch.clamp(E4M3_HALF * (want.abs() + err), min=2.0 ** -10) + err
                if not turn:
                    assert torch.equal(got, want.to(torch.float8_e4m3fn).double())
            assert ((got - want).abs() <= bound).all()
            # nothing else changed
            rest = bits(cache).clone()
            rest[at] = bits(before)[at]
            assert torch.equal(rest, bits(before).view(rest.dtype))
        assert binding.attn_cache_status() == binding.ATTN_OK


@pytest.mark.parametrize("d,begin,dim", [((64, 64), 0, 64), ((128, 128), 0, 128),
                                         ((128, 128), 32, 64), ((192, 128), 128, 64),
                                         ((128, 128), 0, 0)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("order,page,inter", [("token", 16, False), ("head", 7, True),
                                              ("joint", 1, False), ("token", 64, True)])
def test_ragged(d, begin, dim, kind, order, page, inter):
    c = Case(d, kind, order, page, past=[0, 5, 63, 64, 200], new=[3, 1, 2, 0, 90], begin=begin,
             dim=dim, inter=inter)
    c.check(c.append())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 4])
@pytest.mark.parametrize("hq,heads", [(1, 1), (6, 3), (32, 8)])
def test_the_same_number_each(kind, new, hq, heads):
    c = Case((128, 128), kind, "token", 16, past=[0, 15, 16, 17, 1000], new=[new] * 5, hq=hq,
             heads=heads, dim=128, scales=False)
    assert c.cu is None
    c.check(c.append())


def test_far_positions_and_long_prompts():
    c = Case((64, 64), "bf16", "token", 256, past=[1 << 18], new=[2000], dim=64)
    c.check(c.append())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,hq,heads,dim,past,new", [
    ((64, 64), 1, 1, 64, [5, 0, 7, 100], [40000, 3, 0, 31007]),   # many rows side by side
    ((64, 64), 2, 1, 0, [5, 0], [30000, 3001]),                   # no rotation
    ((128, 128), 130, 2, 128, [3, 0], [2000, 1501]),              # more units than a block has
    ((128, 128), 100, 20, 96, [0], [2501]),                       # threads, and nearly so
    ((192, 128), 16, 16, 64, [777, 0, 1], [3001, 2000, 1])])
def test_long_walks_over_the_rows(kind, d, hq, heads, dim, past, new):
    c = Case(d, kind, "token", 64, past, new, hq=hq, heads=heads, begin=d[0] - dim if dim else 0,
             dim=dim, inter=d[0] == 192)
    c.check(c.append())
    q = c.q.clone()
    got = c.append(q_out=c.q).clone()  # in place
    c.q = q
    c.check(got)


def test_without_queries_and_in_place():
    c = Case((128, 128), "bf16", "token", 16, past=[3, 9], new=[1, 1], dim=128)
    assert binding.cache_append(c.cache, c.k, c.v, c.table, c.lens_t(), rotation=c.rot) is None
    c.check(c.turned(c.q)[0])  # (the queries' own form stands in: there are none)
    c = Case((128, 128), "bf16", "token", 16, past=[3, 9], new=[1, 1], dim=128)
    q = c.q.clone()
    assert c.append(q_out=c.q) is c.q
    got = c.q.clone()
    c.q = q
    c.check(got)


@pytest.mark.parametrize("cu", [None, [0, 1, 2, 3, 4]])
def test_unused_rows_are_left_alone(cu):
    """Sequences of length 0, as in a padded batch: their tokens write nothing, q_out included,
    and their table rows are not read."""
    c = Case((64, 64), "bf16", "token", 16, past=[3, 5, 40, 0], new=[1, 1, 1, 1], dim=64)
    q_out = torch.full_like(c.q, 7.0).contiguous()
    lens = c.lens_t()
    lens[1] = 0
    lens[3] = 0
    table = c.table.clone()
    table[1] = 10 ** 9
    table[3] = -5
    binding.cache_append(c.cache, c.k, c.v, table, lens, q=c.q, rotation=c.rot, cu_seqlens=cu,
                         q_out=q_out)
    assert (q_out[[1, 3]] == 7).all()
    used = torch.tensor([True, False, True, False]).cuda()
    want, mag = c.turned(c.q)
    q_out[~used] = want[~used].to(torch.bfloat16)
    c.check(q_out, written=used)


@pytest.mark.parametrize("cu", [None, [0, 0, 0]])
def test_a_step_without_new_tokens(cu):
    c = Case((64, 64), "bf16", "token", 16, [3, 5], [1, 1], dim=64)
    none = [x[:0].contiguous() for x in (c.k, c.v, c.q)]
    got = binding.cache_append(c.cache, none[0], none[1], c.table, c.lens_t(), q=none[2],
                               rotation=c.rot, cu_seqlens=cu)
    assert got.shape == (0, 4, 64)
    assert binding.cache_append(c.cache, none[0], none[1], c.table, c.lens_t()) is None
    assert torch.equal(bits(c.kc), bits(c.before[0])) and torch.equal(bits(c.vc), bits(c.before[1]))


def test_fewer_cached_than_new():
    """lens below the number of new tokens: the ones in front of position 0 are ignored."""
    c = Case((64, 64), "bf16", "token", 16, past=[0], new=[5], dim=64)
    lens = torch.tensor([3], dtype=torch.int32).cuda()
    q_out = torch.full_like(c.q, 7.0).contiguous()
    binding.cache_append(c.cache, c.k, c.v, c.table, lens, q=c.q, rotation=c.rot, q_out=q_out)
    assert (q_out[:2] == 7).all()
    c.pos = torch.tensor([-2, -1, 0, 1, 2]).cuda()
    want, _ = c.turned(c.q)
    q_out[:2] = want[:2].to(torch.bfloat16)
    c.check(q_out, written=c.pos >= 0)


@pytest.mark.parametrize("bad", [-1, -2, -2 ** 31, 2 ** 31 - 1, "pages"])
def test_bad_pages_write_nothing(bad):
    c = Case((128, 128), "bf16", "token", 16, past=[0, 20, 5], new=[30, 1, 20], dim=128)
    table = c.table.clone()
    table[0, 1] = c.kc.shape[0] if bad == "pages" else bad
    q_out = binding.cache_append(c.cache, c.k, c.v, table, c.lens_t(), q=c.q, rotation=c.rot,
                                 cu_seqlens=c.cu)
    assert binding.attn_cache_status() == binding.ATTN_ERR_BAD_PAGE
    # tokens 16 .. 29 of sequence 0 are on that page
    c.check(q_out, written=~((c.seq == 0) & (c.pos >= 16)))


def test_length_past_the_table():
    c = Case((64, 64), "e4m3", "token", 8, past=[10, 0], new=[1, 1], dim=64)
    lens = c.lens_t()
    lens[0] = c.table.shape[1] * 8 + 1
    binding.cache_append(c.cache, c.k, c.v, c.table, lens, rotation=c.rot)
    assert binding.attn_cache_status() == binding.ATTN_ERR_BAD_PAGE
    assert binding.attn_cache_status() == binding.ATTN_OK
    c.check(c.turned(c.q)[0], written=torch.tensor([False, True]).cuda())


def test_e4m3_saturates_and_keeps_nan():
    c = Case((64, 64), "e4m3", "token", 16, past=[0], new=[1], scales=False)
    vals = torch.tensor([448.0, 460.0, 480.0, 1e30, -1e30, float("inf"), float("-inf"),
                         float("nan"), 0.0, -0.0, 2.0 ** -9, 2.0 ** -10, 2.0 ** -11, 17.0, 18.0,
                         19.0]).to(torch.bfloat16).cuda()
    c.k[0, 0, :16] = vals
    c.append()
    got = bits(c.kc)[c.table[0, 0].long(), 0, 0, :16].view(torch.float8_e4m3fn).float()
    want = vals.float().clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert torch.equal(got[:7], want[:7]) and torch.isnan(got[7]) and torch.equal(got[8:], want[8:])


def test_a_cache_beyond_32_bit_offsets():
    """Pages past 2^31 bytes and 2^31 elements."""
    page, heads, d = 64, 8, 128
    pages = 2 ** 31 // (page * heads * d) + 40
    kc = torch.zeros(pages, page, heads, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    cache = binding.PagedCache(kc, vc)
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32).cuda()
    k, v = _rand(1, 70, heads, d), _rand(2, 70, heads, d)
    binding.cache_append(cache, k, v, table, torch.tensor([70], dtype=torch.int32).cuda())
    assert torch.equal(kc[pages - 1], k[:64]) and torch.equal(vc[pages - 1], v[:64])
    assert torch.equal(kc[pages - 3, :6], k[64:]) and torch.equal(vc[pages - 3, :6], v[64:])
    assert kc[pages - 3, 6:].count_nonzero() == 0 and kc[:40].count_nonzero() == 0
    assert kc[pages - 2].count_nonzero() == 0


def test_captured_call_follows_lengths():
    c = Case((64, 64), "bf16", "token", 16, past=[3, 20], new=[1, 1], dim=64)
    table = torch.arange(8, dtype=torch.int32).cuda().view(2, 4)
    kc = make_cache(8, 16, 2, 64, "bf16", "token", 5)
    vc = make_cache(8, 16, 2, 64, "bf16", "token", 6)
    cache = binding.PagedCache(kc, vc)
    lens = c.lens_t()
    q_out = torch.empty_like(c.q).contiguous()
    binding.cache_append(cache, c.k, c.v, table, lens, q=c.q, rotation=c.rot, q_out=q_out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.cache_append(cache, c.k, c.v, table, lens, q=c.q, rotation=c.rot, q_out=q_out)
    lens += 7
    g.replay()
    torch.cuda.synchronize()
    k2 = make_cache(8, 16, 2, 64, "bf16", "token", 5)
    v2 = make_cache(8, 16, 2, 64, "bf16", "token", 6)
    other = binding.PagedCache(k2, v2)
    binding.cache_append(other, c.k, c.v, table, lens - 7, q=c.q, rotation=c.rot)
    want = binding.cache_append(other, c.k, c.v, table, lens, q=c.q, rotation=c.rot)
    assert torch.equal(kc, k2) and torch.equal(vc, v2) and torch.equal(q_out, want)
