"""Cases for measuring grouped prompt attention, prefill over the paged cache, and head norms.

Three families of operators, as a program that trains or serves a model with fewer key heads
than query heads calls them.  ``forward`` / ``backward`` attend whole prompts and packed
training sequences, every key head serving a group of query heads.  ``prefill`` attends a chunk
of new tokens per sequence over a paged cache that holds them already.  ``norm_rope`` scales
each query and key head to unit root mean square and turns it to its position in the same pass,
``norm_rope_backward`` gives the gradients of that, and ``cache_append`` does it on the way into
the cache.

With ``own`` false, ``run`` computes a case in its plain form (elementary torch operations in
fp32, angles in fp64, one rounding at the end); with ``own`` true it makes the library's calls
on the same inputs.
"""
import math

import torch

own = False

_BASE = 10000.0
_EPS = 1e-6


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def _prompt(name, batch, hq, hkv, dqk, dv, short, long, grad, packed=False, window=-1):
    return {"name": name, "op": "prompt", "batch": batch, "hq": hq, "hkv": hkv, "dqk": dqk,
            "dv": dv, "short": short, "long": long, "grad": grad, "packed": packed,
            "window": window}


def _prefill(name, batch, hq, hkv, dqk, dv, new_short, new_long, past_short, past_long, page,
             kind="bf16", order="token", window=-1, idle=0):
    return {"name": name, "op": "prefill", "batch": batch, "hq": hq, "hkv": hkv, "dqk": dqk,
            "dv": dv, "new_short": new_short, "new_long": new_long, "past_short": past_short,
            "past_long": past_long, "page": page, "kind": kind, "order": order,
            "window": window, "idle": idle}


def _norm(name, batch, hq, hkv, d, long, grad, begin, dim, interleaved=False, packed=True,
          pos0=0):
    return {"name": name, "op": "norm", "batch": batch, "hq": hq, "hkv": hkv, "d": d,
            "long": long, "grad": grad, "begin": begin, "dim": dim, "interleaved": interleaved,
            "packed": packed, "pos0": pos0}


def _append(name, batch, hq, hkv, dqk, dv, new_short, new_long, past, page, kind="bf16",
            order="token", begin=0, dim=0, interleaved=False):
    return {"name": name, "op": "append", "batch": batch, "hq": hq, "hkv": hkv, "dqk": dqk,
            "dv": dv, "new_short": new_short, "new_long": new_long, "past": past, "page": page,
            "kind": kind, "order": order, "begin": begin, "dim": dim,
            "interleaved": interleaved}


def listed():
    return [
        # one short prompt through a small model: all latency
        _prompt("prompt_short", 1, 8, 2, 64, 64, 77, 77, False),
        # ragged prompts of a serving batch, from the slices of one projection
        _prompt("prompts_ragged", 4, 32, 8, 128, 128, 33, 3501, False, packed=True),
        # the GPT-2-shaped training layer with a third of its key heads
        _prompt("train_layer_d64", 8, 12, 4, 64, 64, 1024, 1024, True, packed=True),
        # long-context training
        _prompt("train_long", 1, 32, 8, 128, 128, 8192, 8192, True),
        # packed training sequences with a sliding window and (192, 128) heads
        _prompt("train_d192_window", 5, 16, 4, 192, 128, 301, 4096, True, window=1023),
        # a few drafted tokens of every sequence checked against its cache
        _prefill("prefill_verify", 32, 32, 8, 128, 128, 5, 5, 33, 8190, 64),
        # one chunk of a long prompt: the largest computation over the cache
        _prefill("prefill_chunk", 1, 32, 8, 128, 128, 2048, 2048, 30011, 30011, 16),
        # single tokens and chunks in one batch, over an 8-bit cache
        _prefill("prefill_mixed_e4m3", 8, 32, 8, 128, 128, 1, 513, 200, 8001, 64, kind="e4m3"),
        # a short question about a very long text: all parallelism comes from its length
        _prefill("prefill_long", 1, 16, 2, 128, 128, 16, 16, 250007, 250007, 128),
        # a training layer's queries and keys, and their gradients
        _norm("norm_rope_train", 2, 32, 8, 128, 8192, False, 0, 128),
        _norm("norm_rope_grad", 2, 32, 8, 128, 8192, True, 0, 128),
        # one decoding step's new tokens
        _append("append_norm_step", 64, 32, 8, 128, 128, 1, 1, 5000, 64, dim=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 250.0)


def _scores(c):
    """Scores that the plain form holds at once."""
    if c["op"] == "prompt":
        return c["batch"] * c["hq"] * c["long"] ** 2
    if c["op"] == "prefill":
        return c["batch"] * c["hq"] * c["new_long"] * (c["new_long"] + c["past_long"])
    return 0


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    most["append"] = most["norm"]
    while True:
        c = _draw_any(rng)
        del c["name"]
        if _scores(c) <= 32 * 8192 ** 2 and _cost(c) <= most[c["op"]]:
            return c


def _draw_any(rng):
    dqk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 12, 16])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 64, 128, 256])
    kind = rng.choice(["bf16", "bf16", "e4m3"])
    order = rng.choice(["token", "token", "head"])
    interleaved = rng.random() < 0.5
    if dqk == 192:
        begin, dim = 128, 64
    else:
        begin, dim = 0, rng.choice([dqk, dqk, dqk // 2])
    window = rng.choice([-1, -1, -1, 0, 127, 1000])
    op = rng.choice(["prompt", "prompt", "prefill", "prefill", "norm", "append"])
    if op == "prompt":
        # (where every row sees its own key alone the gradients of q and k are zero, and what is
        # left of their sums is rounding, which no two computations have alike)
        grad = rng.random() < 0.6
        batch = _log(rng, 1, 16)
        long = _log(rng, 2 if grad else 1, 8192)
        short = long if rng.random() < 0.4 else rng.randint(1, long)
        return _prompt("", batch, hkv * group, hkv, dqk, dv, short, long, grad,
                       rng.random() < 0.5, 31 if grad and window == 0 else window)
    if op == "prefill":
        batch = _log(rng, 1, 96)
        new = _log(rng, 1, 4096)
        past = _log(rng, 1, 150000) - 1
        return _prefill("", batch, hkv * group, hkv, dqk, dv,
                        new if rng.random() < 0.4 else rng.randint(1, new), new,
                        past if rng.random() < 0.4 else rng.randint(0, past), past, page, kind,
                        order, window, rng.choice([0, 0, 1]) if batch > 2 else 0)
    if op == "norm":
        return _norm("", _log(rng, 1, 16), rng.choice([1, 4, 12, 16, 32]), hkv, dqk,
                     _log(rng, 1, 16384), rng.random() < 0.5, begin, dim, interleaved,
                     rng.random() < 0.5, rng.choice([0, 0, 4095, 1000003]))
    batch = _log(rng, 1, 192)
    long = 1 if rng.random() < 0.4 else _log(rng, 2, 4000)
    return _append("", batch, hkv * group, hkv, dqk, dv, rng.randint(1, long), long,
                   rng.randint(0, 2500), page, kind, order, begin, dim, interleaved)


# ----------------------------------------------------------------------------
# Sizes that a case fixes
# ----------------------------------------------------------------------------
def _spread(n, short, long):
    """n lengths spread evenly from short to long (their sum does not depend on a seed)."""
    if n == 1:
        return [long]
    return [short + (long - short) * i // (n - 1) for i in range(n)]


def _new_past(c):
    """New and earlier tokens of each sequence; an idle one brings tokens, and has length 0."""
    live = c["batch"] - c["idle"]
    new = _spread(c["batch"], c["new_short"], c["new_long"])
    past = list(reversed(_spread(live, c["past_short"], c["past_long"])))
    return new, past + [-1] * c["idle"]


def _pairs(n, past, window):
    """Query-key pairs seen by the last n of past + n positions."""
    if window < 0:
        return n * past + n * (n + 1) // 2
    full = max(0, min(n, window - past))  # queries that the window cuts nothing from
    return full * past + full * (full + 1) // 2 + (n - full) * (window + 1)


def work(case):
    c = case
    if c["op"] == "prompt":
        lens = _spread(c["batch"], c["short"], c["long"])
        t, pairs = sum(lens), sum(_pairs(n, 0, c["window"]) for n in lens)
        d = c["dqk"] + c["dv"]
        io = t * (c["hq"] + c["hkv"]) * d * 2
        flops = 2.0 * pairs * c["hq"] * d
        if c["grad"]:
            io = 2 * io + t * c["hq"] * c["dv"] * 2
            flops += 2.0 * pairs * c["hq"] * (3 * c["dqk"] + 2 * c["dv"])
        return {"bytes": io + t * c["hq"] * 4, "flops": flops}
    if c["op"] == "prefill":
        e = 1 if c["kind"] == "e4m3" else 2
        new, past = _new_past(c)
        d, w = c["dqk"] + c["dv"], c["window"]
        live = [(n, p) for n, p in zip(new, past) if p >= 0]
        keys = sum(n + min(p, w) if w >= 0 else n + p for n, p in live)
        pairs = sum(_pairs(n, p, w) for n, p in live)
        return {"bytes": keys * c["hkv"] * d * e + sum(new) * c["hq"] * (2 * d + 4),
                "flops": 2.0 * pairs * c["hq"] * d}
    if c["op"] == "norm":
        t = c["batch"] * c["long"] * (c["hq"] + c["hkv"])
        passes = 3 if c["grad"] else 2
        return {"bytes": t * c["d"] * 2 * passes, "flops": (14.0 if c["grad"] else 7.0) * t * c["d"]}
    e = 1 if c["kind"] == "e4m3" else 2
    t = sum(_spread(c["batch"], c["new_short"], c["new_long"]))
    return {"bytes": t * (c["hkv"] * (c["dqk"] + c["dv"]) * (2 + e) + c["hq"] * c["dqk"] * 4),
            "flops": 7.0 * t * (c["hq"] + c["hkv"]) * c["dqk"]}


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


def _offsets(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def _projection(rand, shape, heads, together):
    """Tensors shape + (H, d) for each (H, d): slices of one projection, or each its own."""
    if not together:
        return [rand(*shape, h, d) for h, d in heads]
    row = rand(*shape, sum(h * d for h, d in heads))
    parts = row.split([h * d for h, d in heads], -1)
    return [p.unflatten(-1, hd) for p, hd in zip(parts, heads)]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    s = {"case": c}
    if c["op"] == "prompt":
        lens = _spread(c["batch"], c["short"], c["long"])
        even = c["short"] == c["long"]
        shape = (c["batch"], c["long"]) if even else (sum(lens),)
        heads = [(c["hq"], c["dqk"]), (c["hkv"], c["dqk"]), (c["hkv"], c["dv"])]
        s["q"], s["k"], s["v"] = _projection(rand, shape, heads, c["packed"])
        if c["grad"]:
            s["dO"] = rand(*shape, c["hq"], c["dv"])
        s["scale"] = 1.0 / math.sqrt(c["dqk"])
        s["cu"] = None if even else _offsets(lens)
        s["lens"] = lens
        s["length"] = torch.tensor(lens, device="cuda")
        return s

    if c["op"] in ("norm", "append"):
        s["inv_freq"] = torch.tensor([_BASE ** (-2.0 * i / c["dim"])
                                      for i in range(c["dim"] // 2)],
                                     dtype=torch.float64, device="cuda")
        d = c["d"] if c["op"] == "norm" else c["dqk"]
        weight = lambda: 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["q_weight"], s["k_weight"] = weight(), weight()
    if c["op"] == "norm":
        shape = (c["batch"], c["long"])
        heads = [(c["hq"], c["d"]), (c["hkv"], c["d"])]
        s["q"], s["k"] = (x * 1.5 for x in _projection(rand, shape, heads, False)) \
            if not c["packed"] else _projection(rand, shape, heads + [heads[1]], True)[:2]
        if c["grad"]:
            s["dq"], s["dk"] = _projection(rand, shape, heads, False)
        s["pos"] = torch.arange(c["long"], device="cuda") + c["pos0"]
    else:
        if c["op"] == "prefill":
            new, past = _new_past(c)
        else:
            new = _spread(c["batch"], c["new_short"], c["new_long"])
            past = list(reversed(_spread(c["batch"], 0, c["past"])))
        mixed = torch.randperm(c["batch"], generator=g, device="cuda").cpu().tolist()
        new, past = [new[i] for i in mixed], [past[i] for i in mixed]
        lens = [n + p if p >= 0 else 0 for n, p in zip(new, past)]
        s["cu"] = _offsets(new)
        s["offsets"] = None if c["new_short"] == c["new_long"] else s["cu"]
        s["table"], pages = _tables(g, lens, c["page"])
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k_cache"] = _cache(g, pages, c["page"], c["hkv"], c["dqk"], c["kind"], c["order"])
        s["v_cache"] = _cache(g, pages, c["page"], c["hkv"], c["dv"], c["kind"], c["order"])
        s["k_scale"] = s["v_scale"] = None
        if c["kind"] == "e4m3":  # the size of one stored unit, per key head
            unit = lambda: (1 + torch.rand(c["hkv"], generator=g, device="cuda")) / 48
            s["k_scale"], s["v_scale"] = unit(), unit()
        t = s["cu"][-1]
        s["seq"] = torch.repeat_interleave(torch.arange(c["batch"]), torch.tensor(new)).cuda()
        start = torch.tensor([n - e for n, e in zip(lens, s["cu"][1:])]).cuda()
        s["pos"] = start[s["seq"]] + torch.arange(t, device="cuda")
        if c["op"] == "prefill":
            s["q"] = rand(t, c["hq"], c["dqk"]) * 1.5
            s["scale"] = 1.0 / math.sqrt(c["dqk"])
        else:
            heads = [(c["hq"], c["dqk"]), (c["hkv"], c["dqk"]), (c["hkv"], c["dv"])]
            s["q"], s["k"], s["v"] = _projection(rand, (t,), heads, True)
    if own:
        from attention_backward_flashattention_gb300 import binding
        if c["op"] != "norm":
            s["cache"] = binding.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"],
                                            s["v_scale"])
        if c["op"] == "prefill":
            s["workspace"] = binding.prefill_workspace(s["q"].device)
        else:
            s["rot"] = binding.Rotation(s["inv_freq"], begin=c["begin"],
                                        interleaved=c["interleaved"])
            s["norm"] = binding.HeadNorm(s["q_weight"], s["k_weight"], eps=_EPS)
    return s


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        from attention_backward_flashattention_gb300 import binding
    if c["op"] == "prompt":
        if not own:
            return _plain_prompt(s, c)
        window = None if c["window"] < 0 else (c["window"], 0)
        o, lse = binding.forward(s["q"], s["k"], s["v"], causal=True, scale=s["scale"],
                                 cu_seqlens=s["cu"], window=window)
        if not c["grad"]:
            return o, lse
        return (o, lse) + tuple(binding.backward(
            s["q"], s["k"], s["v"], o, s["dO"], lse, causal=True, scale=s["scale"],
            cu_seqlens=s["cu"], window=window))
    if c["op"] == "prefill":
        if not own:
            return _plain_prefill(s, c)
        return binding.prefill(s["cache"], s["q"], s["table"], s["lens"], scale=s["scale"],
                               window_left=c["window"], cu_seqlens=s["offsets"],
                               workspace=s["workspace"])
    if c["op"] == "norm":
        if not own:
            return _plain_norm_grad(s, c) if c["grad"] else _plain_norm(s, c)
        if c["grad"]:
            return binding.norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["norm"],
                                              s["rot"], pos0=c["pos0"])
        return binding.norm_rope(s["q"], s["k"], s["norm"], s["rot"], pos0=c["pos0"])
    if own:
        q = binding.cache_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], q=s["q"],
                                 rotation=s["rot"], cu_seqlens=s["offsets"], norm=s["norm"])
    else:
        q = _plain_append(s, c)
    return q, s["k_cache"], s["v_cache"]


def _softmax(x, seen):
    """Weights of the seen scores (not yet divided), their sum, and the log-sum-exp."""
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    return p, total, top + torch.log(total)


def _plain_prompt(s, c):
    """Sequences padded to the longest; scores (B, key head, group, query, key)."""
    L = c["long"]
    at = torch.arange(L, device="cuda")
    live = at < s["length"][:, None]

    def padded(x):
        x = x.float()
        if s["cu"] is None:
            return x
        y = torch.zeros((c["batch"], L) + x.shape[1:], device="cuda")
        y[live] = x
        return y

    flat = lambda x: x if s["cu"] is None else x[live]
    heads = lambda x: padded(x).unflatten(2, (c["hkv"], -1)).permute(0, 2, 3, 1, 4)
    back = lambda x: flat(x.permute(0, 3, 1, 2, 4).flatten(2, 3)).to(torch.bfloat16)
    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])
    seen = at <= at[:, None]
    if c["window"] >= 0:
        seen = seen & (at >= at[:, None] - c["window"])
    p, total, lse = _softmax((q @ k.transpose(-1, -2)) * s["scale"], seen)
    p /= total
    o = p @ v
    stat = lse.flatten(1, 2)[..., 0]
    if s["cu"] is not None:
        stat = stat.transpose(1, 2)[live].t().contiguous()
    out = (back(o), stat)
    if not c["grad"]:
        return out
    dO = heads(s["dO"])
    dv = (p.transpose(-1, -2) @ dO).sum(2, keepdim=True)
    ds = dO @ v.transpose(-1, -2)
    ds -= (dO * o).sum(-1, keepdim=True)
    ds *= p
    dq = (ds @ k) * s["scale"]
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True) * s["scale"]
    return out + (back(dq), back(dk), back(dv))


def _gathered(cache, scale, page, offset, kind):
    """(B, L, H, d) rows of a paged cache in fp32."""
    if kind == "bf16":
        return cache[page, offset].float()
    rows = cache.view(torch.uint8)[page, offset].view(torch.float8_e4m3fn).float()
    return rows * scale[:, None]


def _plain_prefill(s, c):
    """Queries and keys padded to the longest of the batch."""
    group, n = c["hq"] // c["hkv"], c["new_long"]
    row = torch.arange(s["cu"][-1], device="cuda") - torch.tensor(s["cu"], device="cuda")[s["seq"]]
    q = torch.zeros(c["batch"], n, c["hq"], c["dqk"], device="cuda")
    q[s["seq"], row] = s["q"].float()
    pos = torch.full((c["batch"], n), -1, device="cuda")
    pos[s["seq"], row] = s["pos"]
    j = torch.arange(c["past_long"] + n, device="cuda")
    seen = j <= pos[..., None]
    if c["window"] >= 0:
        seen &= j >= pos[..., None] - c["window"]
    page = s["table"].long()[:, (j // c["page"]).clamp(max=s["table"].shape[1] - 1)].clamp(min=0)
    offset = (j % c["page"]).expand_as(page)
    k = _gathered(s["k_cache"], s["k_scale"], page, offset, c["kind"]).permute(0, 2, 3, 1)
    q = q.unflatten(2, (c["hkv"], group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = (q @ k) * s["scale"]
    del k
    p, total, lse = _softmax(x.unflatten(2, (group, n)), seen[:, None, None])
    del x
    v = _gathered(s["v_cache"], s["v_scale"], page, offset, c["kind"]).permute(0, 2, 1, 3)
    o = (p.flatten(2, 3) @ v).unflatten(2, (group, n)) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["seq"], row]
    lse = lse[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[s["seq"], row]
    return o.to(torch.bfloat16), lse


def _angles(s, sign=1.0):
    """cos and sin (T, 1, dim/2) of the positions' angles."""
    a = sign * s["pos"].double()[:, None] * s["inv_freq"]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotated(x, cos, sin, c):
    """x (..., T, H, d) in fp32 with columns begin .. begin + dim - 1 rotated in pairs."""
    part = x[..., c["begin"]:c["begin"] + c["dim"]]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = part.chunk(2, -1)
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([x[..., :c["begin"]], turned, x[..., c["begin"] + c["dim"]:]], -1)


def _normed(x, weight):
    x = x.float()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS) * weight


def _plain_norm(s, c):
    cos, sin = _angles(s)
    return (_rotated(_normed(s["q"], s["q_weight"]), cos, sin, c).to(torch.bfloat16),
            _rotated(_normed(s["k"], s["k_weight"]), cos, sin, c).to(torch.bfloat16))


def _plain_norm_grad(s, c):
    """dx = r (g - x r^2 mean(g x)) with g = w times the turned-back dy, and dw, sums over all
    rows (of up to a million terms: in 64 bits)."""
    cos, sin = _angles(s, -1.0)

    def side(x, dy, w):
        x, dy = x.float(), _rotated(dy.float(), cos, sin, c)
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)
        g = dy * w
        dx = r * (g - x * (r * r * (g * x).mean(-1, keepdim=True)))
        dw = (dy * x * r).flatten(0, -2).sum(0, dtype=torch.float64).float()
        return dx.to(torch.bfloat16), dw

    dq, dqw = side(s["q"], s["dq"], s["q_weight"])
    dk, dkw = side(s["k"], s["dk"], s["k_weight"])
    return dq, dk, dqw, dkw


def _stored(x, scale, kind):
    """What the cache keeps of x (T, H, d), as bf16 or e4m3 bits."""
    if kind == "bf16":
        return x.to(torch.bfloat16)
    units = x.double() / scale.double()[:, None]  # in 64 bits: values next to a border
    return units.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s, c):
    cos, sin = _angles(s)
    q = _rotated(_normed(s["q"], s["q_weight"]), cos, sin, c).to(torch.bfloat16)
    k = _rotated(_normed(s["k"], s["k_weight"]), cos, sin, c)
    page = s["table"][s["seq"], s["pos"] // c["page"]].long()
    at = (page, s["pos"] % c["page"])
    bits = (lambda t: t.view(torch.uint8)) if c["kind"] == "e4m3" else (lambda t: t)
    bits(s["k_cache"])[at] = _stored(k, s["k_scale"], c["kind"])
    bits(s["v_cache"])[at] = _stored(s["v"].float(), s["v_scale"], c["kind"])
    return q


# ----------------------------------------------------------------------------
# The definition in 64 bits
# ----------------------------------------------------------------------------
def _turn64(x, pos, c):
    """Rotation of x (T, H, d) as a product of complex numbers, in fp64."""
    half = c["dim"] // 2
    rate = torch.arange(half, dtype=torch.float64, device="cuda") * (-math.log(_BASE) / half)
    angle = pos.double()[:, None] * torch.exp(rate)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    cols = torch.arange(c["begin"], c["begin"] + c["dim"], device="cuda")
    pairs = cols.view(half, 2).T if c["interleaved"] else cols.view(2, half)
    z = torch.complex(x[..., pairs[0]], x[..., pairs[1]]) * turn
    y = x.clone()
    y[..., pairs[0]], y[..., pairs[1]] = z.real, z.imag
    return y


def _unit64(x, weight):
    return weight * x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)


def _attend64(q, k, v, scale, first, window):
    """O and LSE of queries (G, n, d) at positions first .. over keys (L, d), in fp64."""
    n, L = q.shape[1], k.shape[0]
    x = q @ k.T * scale
    hidden = torch.ones(n, L, dtype=torch.bool, device="cuda").triu(first + 1)
    if window >= 0:
        hidden |= torch.ones_like(hidden).tril(first - window - 1)
    x = x.masked_fill(hidden, -math.inf)
    return torch.softmax(x, -1) @ v, torch.logsumexp(x, -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "prompt":
        return _exact_prompt(c, s)
    if c["op"] == "prefill":
        return _exact_prefill(c, s)
    pos = s["pos"].repeat(c["batch"]) if c["op"] == "norm" else s["pos"]
    flat = lambda x: x.reshape(-1, x.shape[-2], x.shape[-1]).double()
    if c["op"] == "norm" and c["grad"]:
        outs, weights = [], []
        for n in ("q", "k"):  # by differentiation of the definition
            x = flat(s[n]).requires_grad_()
            w = s[n + "_weight"].double().requires_grad_()
            _turn64(_unit64(x, w), pos, c).backward(flat(s["d" + n]))
            outs.append(x.grad.view(s[n].shape))
            weights.append(w.grad)
        return tuple(outs + weights)
    q, k = (_turn64(_unit64(flat(s[n]), s[n + "_weight"].double()), pos, c) for n in ("q", "k"))
    if c["op"] == "norm":
        return q.view(s["q"].shape), k.view(s["k"].shape)
    new, out = {"k": k, "v": s["v"].double()}, [q]
    for n in ("k", "v"):
        cache, units = s[n + "_cache"].double(), new[n]
        if c["kind"] == "e4m3":
            units = (units / s[n + "_scale"].double()[:, None]).clamp(-448, 448)
        slot = s["table"].long()[s["seq"], pos // c["page"]]
        cache[slot, pos % c["page"]] = units
        out.append(cache)
    return tuple(out)


def _exact_prompt(c, s):
    group = c["hq"] // c["hkv"]
    flat = lambda x: x.flatten(0, 1) if s["cu"] is None else x
    rows = {n: flat(s[n]) for n in ("q", "k", "v", "dO") if n in s}
    t = rows["q"].shape[0]
    o = torch.zeros(t, c["hq"], c["dv"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["hq"], t, dtype=torch.float64, device="cuda")
    grads = {n: torch.zeros(rows[n].shape, dtype=torch.float64, device="cuda")
             for n in ("q", "k", "v")}
    cu = _offsets(s["lens"])
    for b in range(c["batch"]):
        r = slice(cu[b], cu[b + 1])
        for h in range(c["hkv"]):
            hs = slice(h * group, (h + 1) * group)
            q = rows["q"][r, hs].double().transpose(0, 1).requires_grad_(c["grad"])
            k, v = (rows[n][r, h].double().requires_grad_(c["grad"]) for n in ("k", "v"))
            oh, lh = _attend64(q, k, v, s["scale"], 0, c["window"])
            o[r, hs], lse[hs, r] = oh.detach().transpose(0, 1), lh.detach()
            if c["grad"]:  # by differentiation of the definition
                oh.backward(rows["dO"][r, hs].double().transpose(0, 1))
                grads["q"][r, hs] = q.grad.transpose(0, 1)
                grads["k"][r, h], grads["v"][r, h] = k.grad, v.grad
    shaped = lambda x: x if s["cu"] is not None else x.unflatten(0, (c["batch"], c["long"]))
    if s["cu"] is None:
        lse = lse.unflatten(1, (c["batch"], c["long"])).transpose(0, 1)
    out = (shaped(o), lse)
    return out + tuple(shaped(grads[n]) for n in ("q", "k", "v")) if c["grad"] else out


def _exact_prefill(c, s):
    group = c["hq"] // c["hkv"]
    t = s["cu"][-1]
    o = torch.zeros(t, c["hq"], c["dv"], dtype=torch.float64, device="cuda")
    lse = torch.full((t, c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        r = slice(s["cu"][b], s["cu"][b + 1])
        first = n - (r.stop - r.start)
        j = torch.arange(n, device="cuda")
        at = (s["table"][b].long()[j // c["page"]], j % c["page"])
        if c["kind"] == "e4m3":
            k, v = (s[m].view(torch.uint8)[at].view(torch.float8_e4m3fn)
                    for m in ("k_cache", "v_cache"))
        else:
            k, v = s["k_cache"][at], s["v_cache"][at]
        for h in range(c["hkv"]):
            kh, vh = k[:, h].double(), v[:, h].double()
            if c["kind"] == "e4m3":
                kh, vh = kh * s["k_scale"][h].double(), vh * s["v_scale"][h].double()
            hs = slice(h * group, (h + 1) * group)
            q = s["q"][r, hs].double().transpose(0, 1)
            oh, lh = _attend64(q, kh, vh, s["scale"], first, c["window"])
            o[r, hs], lse[r, hs] = oh.transpose(0, 1), lh.t()
    return o, lse
