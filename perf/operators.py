"""Cases for measuring the rotation, cache-append and decode operators.

Three operators, as a program that trains or serves with this library calls
them.  ``rope`` rotates queries and keys by their positions before the forward
(and, inverted, their gradients after the backward).  ``append`` writes the new
tokens' keys and values into a paged cache, with the rotation applied on the
way, and returns the rotated queries.  ``decode`` is the attention of one new
token per sequence over that cache.

With ``own`` false, ``run`` computes a case in its plain form (elementary torch
operations in fp32, angles in fp64, one rounding at the end); with ``own`` true
it makes the library's calls on the same inputs.
"""
import math

import torch

own = False

_BASE = 10000.0


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def _decode(name, batch, hq, hkv, dqk, dv, short, long, page, kind="bf16", order="token",
            window=-1, idle=0):
    return {"name": name, "op": "decode", "batch": batch, "hq": hq, "hkv": hkv, "dqk": dqk,
            "dv": dv, "short": short, "long": long, "page": page, "kind": kind, "order": order,
            "window": window, "idle": idle}


def _append(name, batch, hq, hkv, dqk, dv, new_short, new_long, past, page, kind="bf16",
            order="token", begin=0, dim=0, interleaved=False):
    return {"name": name, "op": "append", "batch": batch, "hq": hq, "hkv": hkv, "dqk": dqk,
            "dv": dv, "new_short": new_short, "new_long": new_long, "past": past, "page": page,
            "kind": kind, "order": order, "begin": begin, "dim": dim,
            "interleaved": interleaved}


def _rope(name, batch, hq, hk, d, short, long, begin, dim, interleaved=False, inverse=False,
          packed=False, pos0=0):
    return {"name": name, "op": "rope", "batch": batch, "hq": hq, "hk": hk, "d": d,
            "short": short, "long": long, "begin": begin, "dim": dim,
            "interleaved": interleaved, "inverse": inverse, "packed": packed, "pos0": pos0}


def listed():
    return [
        # one short conversation's next token: all latency
        _decode("decode_short", 1, 16, 16, 128, 128, 130, 130, 16),
        # the GPT-2-shaped layer generating at half its context
        _decode("decode_layer_d64", 8, 12, 12, 64, 64, 1, 1024, 64),
        # a serving batch with grouped heads, ragged lengths and unused rows
        _decode("decode_grouped", 64, 32, 8, 128, 128, 33, 8190, 64, idle=3),
        # one very long context with two key heads: all parallelism comes from its length
        _decode("decode_long", 1, 16, 2, 128, 128, 250007, 250007, 128),
        # a large batch over an 8-bit cache: the largest read
        _decode("decode_e4m3", 128, 64, 8, 128, 128, 1, 16384, 64, kind="e4m3"),
        # the (192, 128) head with head-major pages
        _decode("decode_d192", 16, 16, 16, 192, 128, 500, 4099, 32, order="head"),
        # one decoding step's new tokens, queries rotated on the way
        _append("append_step", 64, 32, 8, 128, 128, 1, 1, 5000, 64, dim=128),
        # ragged prompts entering an 8-bit cache
        _append("append_prompts_e4m3", 12, 32, 8, 128, 128, 301, 2500, 0, 64, kind="e4m3",
                dim=128),
        # the (192, 128) head: the last 64 of 192 rotated, in adjacent pairs, head-major pages
        _append("append_d192", 4, 16, 16, 192, 128, 1024, 4096, 777, 32, order="head",
                begin=128, dim=64, interleaved=True),
        # the GPT-2-shaped training layer's forward, from its packed projection
        _rope("rope_layer_packed", 8, 12, 12, 64, 1024, 1024, 0, 64, packed=True),
        # gradients of queries and keys in long-context training
        _rope("rope_grad_long", 1, 16, 16, 128, 32768, 32768, 0, 128, inverse=True),
        # a ragged batch far into its context, part of each head rotated
        _rope("rope_far_ragged", 7, 16, 4, 192, 513, 8001, 128, 64, interleaved=True,
              pos0=500000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        c = _draw_any(rng)
        del c["name"]
        # the plain form of a decode pads every sequence to the longest
        padded = c["batch"] * c["hkv"] * c["long"] <= 128 * 8 * 16384 if c["op"] == "decode" \
            else True
        if padded and work(c)["bytes"] <= most / 2:
            return c


def _draw_any(rng):
    dqk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 12, 16])
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 8, 12, 16, 24])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 64, 128, 256])
    kind = rng.choice(["bf16", "bf16", "e4m3"])
    order = rng.choice(["token", "token", "head"])
    interleaved = rng.random() < 0.5
    if dqk == 192:
        begin, dim = 128, 64
    else:
        begin, dim = 0, rng.choice([dqk, dqk, dqk // 2])
    op = rng.choice(["decode", "decode", "append", "rope"])
    if op == "decode":
        batch = _log(rng, 1, 192)
        long = _log(rng, 1, 200000)
        short = long if rng.random() < 0.3 else rng.randint(1, long)
        return _decode("", batch, hkv * group, hkv, dqk, dv, short, long, page, kind, order,
                       window=rng.choice([-1, -1, -1, 0, 127, 1000]),
                       idle=rng.choice([0, 0, 1]) if batch > 2 else 0)
    if op == "append":
        batch = _log(rng, 1, 192)
        long = 1 if rng.random() < 0.4 else _log(rng, 2, 6000)
        return _append("", batch, hkv * group, hkv, dqk, dv, rng.randint(1, long), long,
                       rng.randint(0, 3000), page, kind, order, begin, dim, interleaved)
    batch = _log(rng, 1, 16)
    long = _log(rng, 1, 32768)
    packed = rng.random() < 0.4
    hq = rng.choice([1, 4, 12, 16, 16, 32])
    return _rope("", batch, hq, hq if packed else hkv, dqk,
                 long if packed or rng.random() < 0.4 else rng.randint(1, long), long, begin,
                 dim, interleaved, rng.random() < 0.5, packed,
                 rng.choice([0, 0, 4095, 1000003]))


# ----------------------------------------------------------------------------
# Sizes that a case fixes
# ----------------------------------------------------------------------------
def _spread(n, short, long):
    """n lengths spread evenly from short to long (their sum does not depend on a seed)."""
    if n == 1:
        return [long]
    return [short + (long - short) * i // (n - 1) for i in range(n)]


def _lens(c):
    full = _spread(c["batch"] - c["idle"], c["short"], c["long"])
    return full + [0] * c["idle"]


def work(case):
    c = case
    if c["op"] == "decode":
        e = 1 if c["kind"] == "e4m3" else 2
        w = c["window"]
        keys = sum(min(n, w + 1) if w >= 0 else n for n in _lens(c))
        d = c["dqk"] + c["dv"]
        return {"bytes": keys * c["hkv"] * d * e + c["batch"] * c["hq"] * (2 * d + 4),
                "flops": 2.0 * keys * c["hq"] * d}
    if c["op"] == "append":
        e = 1 if c["kind"] == "e4m3" else 2
        t = sum(_spread(c["batch"], c["new_short"], c["new_long"]))
        return {"bytes": t * (c["hkv"] * (c["dqk"] + c["dv"]) * (2 + e) + c["hq"] * c["dqk"] * 4),
                "flops": 3.0 * t * (c["hq"] + c["hkv"]) * c["dim"]}
    t = sum(_spread(c["batch"], c["short"], c["long"]))
    return {"bytes": t * (c["hq"] + c["hk"]) * c["d"] * 4,
            "flops": 3.0 * t * (c["hq"] + c["hk"]) * c["dim"]}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _cache(g, pages, page, heads, d, kind, order):
    """A paged cache tensor indexed (page, token, head, column), holding earlier tokens."""
    shape = (pages, heads, page, d) if order == "head" else (pages, page, heads, d)
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if kind == "e4m3":
        x = (x * 32).to(torch.float8_e4m3fn)
    return x.transpose(1, 2) if order == "head" else x


def _tables(g, lens, page, spare=2):
    """Block table (-1 where a sequence has no page) over shuffled pages, and the page count."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    rows = torch.tensor(need, device="cuda")
    width = max(1, max(need))
    at = torch.arange(width, device="cuda")
    first = torch.cumsum(rows, 0) - rows
    table = ids[(first[:, None] + at).clamp(max=total - 1)]
    return torch.where(at < rows[:, None], table, -1).to(torch.int32).contiguous(), total


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    s = {"case": c}
    if c["op"] in ("append", "rope"):
        s["inv_freq"] = torch.tensor([_BASE ** (-2.0 * i / c["dim"])
                                      for i in range(c["dim"] // 2)],
                                     dtype=torch.float64, device="cuda")
    if c["op"] == "rope":
        lens = _spread(c["batch"], c["short"], c["long"])
        if c["packed"]:
            qkv = rand(c["batch"], c["long"], 3, c["hq"], c["d"])
            s["q"], s["k"] = qkv.select(2, 0), qkv.select(2, 1)
        elif c["short"] == c["long"]:
            s["q"] = rand(c["batch"], c["long"], c["hq"], c["d"])
            s["k"] = rand(c["batch"], c["long"], c["hk"], c["d"])
        else:
            s["q"], s["k"] = rand(sum(lens), c["hq"], c["d"]), rand(sum(lens), c["hk"], c["d"])
            s["cu"] = [sum(lens[:i]) for i in range(len(lens) + 1)]
        s["pos"] = torch.cat([torch.arange(n) for n in lens]).cuda() + c["pos0"]
        if own:
            from attention_backward_flashattention_gb300 import binding
            s["rot"] = binding.Rotation(s["inv_freq"], begin=c["begin"],
                                        interleaved=c["interleaved"])
        return s

    mixed = torch.randperm(c["batch"], generator=g, device="cuda").cpu().tolist()
    if c["op"] == "decode":
        lens = [_lens(c)[i] for i in mixed]
    else:
        new = [_spread(c["batch"], c["new_short"], c["new_long"])[i] for i in mixed]
        past = [_spread(c["batch"], 0, c["past"])[i] for i in reversed(mixed)]
        lens = [a + b for a, b in zip(past, new)]
        s["cu"] = [sum(new[:i]) for i in range(len(new) + 1)]
    s["table"], pages = _tables(g, lens, c["page"])
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["k_cache"] = _cache(g, pages, c["page"], c["hkv"], c["dqk"], c["kind"], c["order"])
    s["v_cache"] = _cache(g, pages, c["page"], c["hkv"], c["dv"], c["kind"], c["order"])
    s["k_scale"] = s["v_scale"] = None
    if c["kind"] == "e4m3":  # the size of one stored unit, per key head
        unit = lambda: (1 + torch.rand(c["hkv"], generator=g, device="cuda")) / 48
        s["k_scale"], s["v_scale"] = unit(), unit()
    if c["op"] == "decode":
        s["q"] = rand(c["batch"], c["hq"], c["dqk"]) * 1.5
        s["scale"] = 1.0 / math.sqrt(c["dqk"])
    else:
        t = s["cu"][-1]
        # the slices of one projection, as a layer has them
        row = rand(t, c["hq"] * c["dqk"] + c["hkv"] * (c["dqk"] + c["dv"]))
        q, k, v = row.split([c["hq"] * c["dqk"], c["hkv"] * c["dqk"], c["hkv"] * c["dv"]], 1)
        s["q"] = q.unflatten(1, (c["hq"], c["dqk"]))
        s["k"] = k.unflatten(1, (c["hkv"], c["dqk"]))
        s["v"] = v.unflatten(1, (c["hkv"], c["dv"]))
        s["seq"] = torch.repeat_interleave(torch.arange(c["batch"]), torch.tensor(new)).cuda()
        start = torch.tensor([p - s["cu"][i] for i, p in enumerate(past)]).cuda()
        s["pos"] = start[s["seq"]] + torch.arange(t, device="cuda")
    if own:
        from attention_backward_flashattention_gb300 import binding
        s["cache"] = binding.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if c["op"] == "decode":
            s["workspace"] = binding.decode_workspace(s["q"].device)
        else:
            s["rot"] = binding.Rotation(s["inv_freq"], begin=c["begin"],
                                        interleaved=c["interleaved"])
            s["offsets"] = None if c["new_long"] == 1 else s["cu"]
    return s


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if c["op"] == "rope":
        if own:
            from attention_backward_flashattention_gb300 import binding
            return binding.rope(s["q"], s["k"], s["rot"], inverse=c["inverse"], pos0=c["pos0"],
                                cu_seqlens=s.get("cu"))
        return _plain_rope(s, c)
    if c["op"] == "append":
        if own:
            from attention_backward_flashattention_gb300 import binding
            q = binding.cache_append(s["cache"], s["k"], s["v"], s["table"], s["lens"],
                                     q=s["q"], rotation=s["rot"], cu_seqlens=s["offsets"])
        else:
            q = _plain_append(s, c)
        return q, s["k_cache"], s["v_cache"]
    if own:
        from attention_backward_flashattention_gb300 import binding
        return binding.decode(s["cache"], s["q"], s["table"], s["lens"], scale=s["scale"],
                              window_left=c["window"], workspace=s["workspace"])
    return _plain_decode(s, c)


def _rotated(x, angles, c):
    """x (..., H, d) in fp32 with columns begin .. begin + dim - 1 rotated in pairs."""
    x = x.float()
    cos, sin = torch.cos(angles).float(), torch.sin(angles).float()
    cos, sin = cos[..., None, :], sin[..., None, :]
    part = x[..., c["begin"]:c["begin"] + c["dim"]]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = part.chunk(2, -1)
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([x[..., :c["begin"]], turned, x[..., c["begin"] + c["dim"]:]], -1)


def _plain_rope(s, c):
    angles = s["pos"].double()[:, None] * s["inv_freq"]
    if c["inverse"]:
        angles = -angles
    angles = angles.reshape(s["q"].shape[:-2] + (-1,))
    return (_rotated(s["q"], angles, c).to(torch.bfloat16),
            _rotated(s["k"], angles, c).to(torch.bfloat16))


def _stored(x, scale, kind):
    """What the cache keeps of x (T, H, d) in fp32, as bf16 or e4m3 bits."""
    if kind == "bf16":
        return x.to(torch.bfloat16)
    units = x.double() / scale.double()[:, None]  # in 64 bits: values next to a border
    return units.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s, c):
    angles = s["pos"].double()[:, None] * s["inv_freq"]
    q = _rotated(s["q"], angles, c).to(torch.bfloat16)
    k = _stored(_rotated(s["k"], angles, c), s["k_scale"], c["kind"])
    v = _stored(s["v"].float(), s["v_scale"], c["kind"])
    page = s["table"][s["seq"], s["pos"] // c["page"]].long()
    at = (page, s["pos"] % c["page"])
    bits = (lambda t: t.view(torch.uint8)) if c["kind"] == "e4m3" else (lambda t: t)
    bits(s["k_cache"])[at] = k
    bits(s["v_cache"])[at] = v
    return q


def _gathered(cache, scale, page, offset, kind):
    """(B, L, H, d) rows of a paged cache in fp32."""
    if kind == "bf16":
        return cache[page, offset].float()
    rows = cache.view(torch.uint8)[page, offset].view(torch.float8_e4m3fn).float()
    return rows * scale[:, None]


def _plain_decode(s, c):
    j = torch.arange(c["long"], device="cuda")
    n = s["lens"].long()[:, None]
    seen = j < n
    if c["window"] >= 0:
        seen &= j >= n - 1 - c["window"]
    page = s["table"].long()[:, j // c["page"]].clamp(min=0)
    offset = (j % c["page"]).expand_as(page)
    k = _gathered(s["k_cache"], s["k_scale"], page, offset, c["kind"]).permute(0, 2, 3, 1)
    group = c["hq"] // c["hkv"]
    q = s["q"].float().unflatten(1, (c["hkv"], group))
    x = (q @ k) * s["scale"]
    del k
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["v_scale"], page, offset, c["kind"]).permute(0, 2, 1, 3)
    o = (p @ v) / torch.where(total > 0, total, 1.0)
    lse = top + torch.log(total)
    return o.flatten(1, 2).to(torch.bfloat16), lse.flatten(1)


# ----------------------------------------------------------------------------
# The definition in 64 bits
# ----------------------------------------------------------------------------
def _turn64(x, pos, c, sign=1.0):
    """Rotation as a product of complex numbers, in fp64."""
    half = c["dim"] // 2
    rate = torch.arange(half, dtype=torch.float64, device="cuda") * (-math.log(_BASE) / half)
    angle = sign * pos.double()[:, None] * torch.exp(rate)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    y = x.double().clone()
    cols = torch.arange(c["begin"], c["begin"] + c["dim"], device="cuda")
    pairs = cols.view(half, 2).T if c["interleaved"] else cols.view(2, half)
    z = torch.complex(y[..., pairs[0]], y[..., pairs[1]]) * turn
    y[..., pairs[0]], y[..., pairs[1]] = z.real, z.imag
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        sign = -1.0 if c["inverse"] else 1.0
        flat = lambda x: x.reshape(-1, x.shape[-2], x.shape[-1])
        return tuple(_turn64(flat(s[n]), s["pos"], c, sign).view(s[n].shape)
                     for n in ("q", "k"))
    if c["op"] == "append":
        new = {"k": _turn64(s["k"], s["pos"], c), "v": s["v"].double()}
        out = [_turn64(s["q"], s["pos"], c)]
        for n in ("k", "v"):
            cache = s[n + "_cache"].double()
            units = new[n]
            if c["kind"] == "e4m3":
                units = (units / s[n + "_scale"].double()[:, None]).clamp(-448, 448)
            slot = s["table"].long()[s["seq"], s["pos"] // c["page"]]
            cache[slot, s["pos"] % c["page"]] = units
            out.append(cache)
        return tuple(out)
    o = torch.zeros(c["batch"], c["hq"], c["dv"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    group = c["hq"] // c["hkv"]
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        first = max(0, n - 1 - c["window"]) if c["window"] >= 0 else 0
        j = torch.arange(first, n, device="cuda")
        slot = s["table"][b].long()[j // c["page"]]
        at = (slot, j % c["page"])
        if c["kind"] == "e4m3":
            k, v = (s[m].view(torch.uint8)[at].view(torch.float8_e4m3fn)
                    for m in ("k_cache", "v_cache"))
        else:
            k, v = s["k_cache"][at], s["v_cache"][at]
        for h in range(c["hkv"]):
            kh, vh = k[:, h].double(), v[:, h].double()
            if c["kind"] == "e4m3":
                kh, vh = kh * s["k_scale"][h].double(), vh * s["v_scale"][h].double()
            rows = slice(h * group, (h + 1) * group)
            x = s["q"][b, rows].double() @ kh.T * s["scale"]
            lse[b, rows] = torch.logsumexp(x, -1)
            o[b, rows] = torch.softmax(x, -1) @ vh
    return o, lse
