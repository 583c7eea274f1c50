"""Plain 64-bit forms of the rotation, the cache and the decode for the tests
(indexing and elementary arithmetic only; nothing of the library)."""
import math

import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2       # 2^-8: one rounding to bf16
E4M3_HALF = torch.finfo(torch.float8_e4m3fn).eps / 2  # 2^-4: one rounding to e4m3


def inv_freq(dim, base=10000.0):
    return [base ** (-2.0 * i / dim) for i in range(dim // 2)]


def rotate64(x, pos, freq, begin, interleaved, sign=1.0):
    """x (..., T, H, d) rotated at positions pos (T), and |a| + |b| of each column's pair."""
    x = x.double()
    dim = 2 * len(freq)
    ang = sign * pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    cos, sin = torch.cos(ang)[:, None, :], torch.sin(ang)[:, None, :]
    y, mag = x.clone(), torch.zeros_like(x)
    if interleaved:
        ia = torch.arange(begin, begin + dim, 2, device=x.device)
        ib = ia + 1
    else:
        ia = torch.arange(begin, begin + dim // 2, device=x.device)
        ib = ia + dim // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * cos - b * sin
    y[..., ib] = a * sin + b * cos
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def rotation_bound(y, mag):
    """Largest error of a rotated bf16 element: its rounding, and fp32 arithmetic.  The angle
    handed to sincospi is off by at most pi * 2^-24 (the rounding of a fraction of a turn to
    fp32), sin and cos are then within 2^-22, and the two products and their sum round three
    times at 2^-24: together below 2^-20 of |a| + |b|."""
    return BF16_HALF * y.abs() + 2.0 ** -20 * mag * (1 + BF16_HALF)


def make_cache(pages, page, heads, d, kind, order, seed, device="cuda"):
    """A cache tensor (pages, page, heads, d) of random values ("head": head-major memory;
    "joint": the first half of a buffer that holds both)."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    shape = {"token": (pages, page, heads, d), "head": (pages, heads, page, d),
             "joint": (pages, 2, page, heads, d)}[order]
    x = torch.randn(shape, generator=g).to(device)
    x = x.to(torch.bfloat16) if kind == "bf16" else (x * 40).to(torch.float8_e4m3fn)
    if order == "head":
        x = x.transpose(1, 2)
    elif order == "joint":
        x = x[:, 0]
    return x


def bits(t):
    """The raw bits of a bf16 or e4m3 tensor (which indexing can write)."""
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8)


def nan_bits(t):
    return 0x7FC0 if t.dtype == torch.bfloat16 else 0x7F


def make_table(lens, page, seed, spare=3, width=None, device="cuda"):
    """Shuffled pages for sequences of these lengths; -1 where no page is needed."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    ids = torch.randperm(total, generator=g).tolist()
    width = max(1, max(need)) if width is None else width
    rows = []
    for n in need:
        rows.append(ids[:n] + [-1] * (width - n))
        ids = ids[n:]
    return torch.tensor(rows, dtype=torch.int32, device=device), total


def seen_keys(n, window):
    return max(0, n - 1 - window) if window >= 0 else 0


def poison_unseen(cache, table, lens, page, window):
    """NaN in every slot that no sequence sees."""
    keep = torch.zeros(cache.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(seen_keys(n, window), n):
            keep[int(table[b, j // page]), j % page] = True
    raw = bits(cache)
    raw[~keep.to(cache.device)] = nan_bits(cache)


def decode64(q, k_cache, v_cache, table, lens, page, scale, window=-1, k_scale=None,
             v_scale=None, hidden=None):
    """O, LSE and error bounds of both, one sequence at a time in fp64.

    hidden: {sequence: keys that take no part}.  The bounds, per element:
      scores: fp32 sums of d products, each rounding at 2^-23 of the sum of absolute values
        (a tensor core truncates), and the rounding of s x (2^-22 of it, scale and exponent);
        an e4m3 cache also takes the queries in fp16 scaled to a largest value in [1, 2),
        which loses at most 2^-25 of that value per element;
      probabilities: 2^-16 of each (two bf16 roundings), or 2^-11 and 2^-25 (fp16);
        the exponential itself 2^-22;
      the sum over n keys: n 2^-23 of the sum of absolute values;
      O: one rounding to bf16."""
    B, Hq, dqk = q.shape
    heads, dv = k_cache.shape[2], v_cache.shape[3]
    e4m3 = k_cache.dtype != torch.bfloat16
    G = Hq // heads
    o = torch.zeros(B, Hq, dv, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        keys = [j for j in range(seen_keys(n, window), n)
                if hidden is None or j not in hidden.get(b, ())]
        if not keys:
            continue
        j = torch.tensor(keys, device=q.device)
        at = (table[b].long()[j // page], j % page)
        k = bits(k_cache)[at].view(k_cache.dtype).double()
        v = bits(v_cache)[at].view(v_cache.dtype).double()
        if k_scale is not None:
            k = k * k_scale.double()[:, None]
        if v_scale is not None:
            v = v * v_scale.double()[:, None]
        qb = q[b].double().view(heads, G, dqk)
        k, v = k.permute(1, 2, 0), v.permute(1, 0, 2)
        x = qb @ k * scale
        mag = (qb.abs() @ k.abs() * scale).amax(-1)
        lse_b = torch.logsumexp(x, -1)
        p = torch.exp(x - lse_b[..., None])
        ob, ab = p @ v, p @ v.abs()
        dx = (dqk + 2) * 2.0 ** -23 * mag + 2.0 ** -22 * x.abs().amax(-1)
        if e4m3:
            dx = dx + dqk * 2.0 ** -25 * qb.abs().amax(-1) * k.abs().amax() * scale
        rel = 2.0 ** -22 + 2 * dx + len(keys) * 2.0 ** -23
        tol = ab * (rel + (2.0 ** -11 if e4m3 else 2.0 ** -16))[..., None]
        if e4m3:
            tol = tol + 2.0 ** -25 * v.abs().sum(1)[:, None, :]
        o[b], lse[b] = ob.reshape(Hq, dv), lse_b.reshape(Hq)
        tol_o[b] = (BF16_HALF * ob.abs() + tol * (1 + BF16_HALF)).reshape(Hq, dv)
        tol_l[b] = (rel + 2.0 ** -22 * lse_b.abs()).reshape(Hq)
    return o, lse, tol_o, tol_l


def check_decode(got, ref, where=""):
    o, lse = got
    ro, rl, to, tl = ref
    empty = rl == -math.inf
    if lse is not None:
        assert torch.equal(lse.double() == -math.inf, empty), where
        over = ((lse.double() - rl).abs() - tl)[~empty]
        assert over.numel() == 0 or (over <= 0).all(), f"{where}: LSE over by {over.max()}"
    assert torch.isfinite(o).all(), where
    over = (o.double() - ro).abs() - to
    assert (over <= 0).all(), f"{where}: O over by {over.max()} at {over.argmax()}"
