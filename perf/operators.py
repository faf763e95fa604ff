"""Performance cases of the operators around a paged 4-bit key/value cache.

* ``rotary``: rotary positions of queries and keys, forward and gradient.
* ``plan``: block tables, slot maps and positions from request lengths.
* ``store``: keys and values quantised into the cache and read back.
* ``attend``: attention of packed queries over the cache (a decode step, a few
  drafted tokens, a chunk of a prompt).

``run`` computes an operator in its plain form, with elementary torch
operations, or, with ``own`` set, calls this package.  ``exact`` restates it
in 64 bits.

The cache is ``uint8 [pages, kv_heads, page / 16, 18 d]``: tiles of 16 tokens
of one head, each K codes (16 rows of d / 2 bytes), K parameters (16 rows of
d / 64 pairs scale, lowest value in bf16), V codes, V parameters.  Eight
channels make a 32-bit word, the first in the lowest four bits; word 4 j + t of
a K row stands at place t d / 32 + j, word 8 j + g of a V row at g d / 64 + j.
"""
import math

import torch

own = False

GROUP = 64  # channels that share a scale and a lowest value


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of a small batch, far into long contexts: latency
        dict(name="rotary decode", op="rotary", batch=1, heads=32, kv_heads=8, tokens=8, d=128, rot=128, pairs="half",
             direction="forward", dtype="bfloat16", packed=True, reach=131072, factor=8.0),
        # the training shape of the benchmark (B=2 H=16 N=4096 d=128)
        dict(name="rotary train", op="rotary", batch=2, heads=16, kv_heads=16, tokens=4096, d=128, rot=128, pairs="half",
             direction="forward", dtype="bfloat16", packed=False, reach=4096, factor=1.0),
        # gradient of the ragged test shape (B=4 H=16 N=1000 d=64), half of each head rotated, neighbouring pairs
        dict(name="rotary gradient", op="rotary", batch=4, heads=16, kv_heads=16, tokens=1000, d=64, rot=32,
             pairs="interleaved", direction="backward", dtype="bfloat16", packed=False, reach=1000, factor=1.0),
        # a decode step of eight requests
        dict(name="plan decode", op="plan", requests=8, page=64, table=64, held_lo=1, held_hi=4000, prompt=0,
             prompt_every=0, shrink_every=0),
        # a full scheduler step: prompts, decodes, requests that end
        dict(name="plan mixed", op="plan", requests=1023, page=16, table=256, held_lo=0, held_hi=3500, prompt=500,
             prompt_every=16, shrink_every=9),
        # the new token of each request of a decode batch
        dict(name="store decode", op="store", tokens=32, kv_heads=8, d=128, page=64, scattered=True),
        # the prompts of a step
        dict(name="store prompt", op="store", tokens=16384, kv_heads=8, d=128, page=64, scattered=False),
        # one short request: latency
        dict(name="attend one", op="attend", requests=1, heads=16, kv_heads=16, d=64, page=16, len_lo=1000, len_hi=1000,
             new=1, causal=True),
        # a decode batch of ragged lengths, grouped heads
        dict(name="attend decode", op="attend", requests=64, heads=32, kv_heads=8, d=128, page=64, len_lo=200, len_hi=8192,
             new=1, causal=True),
        # few requests with long contexts
        dict(name="attend long", op="attend", requests=3, heads=32, kv_heads=8, d=128, page=64, len_lo=100000,
             len_hi=131072, new=1, causal=True),
        # drafted tokens checked in one pass
        dict(name="attend draft", op="attend", requests=24, heads=16, kv_heads=4, d=64, page=32, len_lo=5, len_hi=4096,
             new=5, causal=True),
        # a chunk of a prompt after the chunks before it
        dict(name="attend chunk", op="attend", requests=2, heads=32, kv_heads=8, d=128, page=64, len_lo=3000, len_hi=16384,
             new=1000, causal=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "plan", "store", "attend", "attend"])
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    if op == "rotary":
        packed = rng.random() < 0.5
        batch = 1 if packed else rng.randint(1, 4)
        tokens = _spread(rng, 1, max(2, min(8192, (1 << 26) // (batch * (heads + kv_heads) * d))))
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, tokens=tokens, d=d,
                    rot=rng.choice([d, d // 2, d // 4, d - 2 * rng.randint(1, 20)]), pairs=rng.choice(["half", "interleaved"]),
                    direction=rng.choice(["forward", "backward"]), dtype=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]),
                    packed=packed, reach=_spread(rng, tokens, 1 << 20), factor=rng.choice([1.0, 4.0, 32.0]))
    if op == "plan":
        page = rng.choice([16, 32, 64, 128])
        requests = _spread(rng, 1, 2048)
        table = max(2, _spread(rng, 64, 8192) // page)
        held = max(1, page * table // 2)
        return dict(op=op, requests=requests, page=page, table=table, held_lo=0, held_hi=held,
                    prompt=rng.randint(1, held), prompt_every=rng.choice([0, 4, 16, 31]), shrink_every=rng.choice([0, 5, 9]))
    if op == "store":
        return dict(op=op, tokens=_spread(rng, 1, 16384), kv_heads=min(kv_heads, 8), d=d, page=rng.choice([16, 32, 64, 128]),
                    scattered=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    new = rng.choice([1, 1, 1, 2, 3, 5, 8, _spread(rng, 9, 1000)])
    top = _spread(rng, max(16, new), 65536)
    # the keys read and the products made stay below the largest listed case's
    requests = _spread(rng, 1, 128)
    while requests > 1 and (requests * kv_heads * top * d > 3 << 27 or requests * heads * new * top * d > 1 << 35):
        requests //= 2
    while heads * new * top * d > 1 << 35:
        top, new = max(16, top // 2), max(1, new // 2)
    return dict(op="attend", requests=requests, heads=heads, kv_heads=kv_heads, d=d, page=page,
                len_lo=max(new, rng.randint(1, top)), len_hi=top, new=new, causal=rng.random() < 0.8)


# ------------------------------------------------------------------ inputs
def _ragged(count, lo, hi):
    """`count` lengths of [lo, hi], the first and the second at the ends."""
    return [hi if b == 0 else lo if b == 1 else lo + int((b * 0.6180339887498949 % 1.0) * (hi - lo + 1)) for b in range(count)]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _frequencies(rot, factor):
    """Rotation per position of each pair, base 10000; for a longer context the
    slow pairs are slowed by `factor`, the fast ones kept, with a ramp between."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if factor > 1.0:
        turns = 8192.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f.cuda(), 1.0 if factor <= 1.0 else 0.1 * math.log(factor) + 1.0


def _quantise(x):
    """Codes, scales and lowest values of x [..., d], groups of 64 channels."""
    x = x.double().unflatten(-1, (-1, GROUP))
    lo = x.amin(-1, keepdim=True)
    span = x.amax(-1, keepdim=True) - lo
    scale = (span / 15.0).bfloat16()
    up = (scale.view(torch.int16) + 1).view(torch.bfloat16)
    scale = torch.where(scale.double() * 15.0 < span, up, scale)
    s = scale.double()
    n = torch.where(s > 0, torch.floor((x - lo) / s.clamp_min(1e-300) + 0.5), 0.0).clamp(0.0, 15.0)
    return n.to(torch.uint8).flatten(-2), torch.cat([scale, lo.bfloat16()], -1)


def _rows(x, values):
    """x [..., d] as rows of the cache: code bytes and parameter bytes."""
    n, par = _quantise(x)
    d = x.shape[-1]
    code = n[..., 0::2] | (n[..., 1::2] << 4)
    shape = (d // 64, 8, 4) if values else (d // 32, 4, 4)
    code = code.unflatten(-1, shape).transpose(-3, -2).flatten(-3)
    return code, par.flatten(-2).contiguous().view(torch.uint8)


def _parts(cache, d):
    """The four parts of a cache's tiles: K codes, K parameters, V codes, V parameters, each [pages, heads, blocks, 16, bytes]."""
    a, b = 8 * d, d
    at = [0, a, a + b, 2 * a + b, 2 * a + 2 * b]
    return [cache[..., at[i]:at[i + 1]].unflatten(-1, (16, -1)) for i in range(4)]


def _values(code, par, values, dtype=torch.float32):
    """The values that rows of the cache stand for."""
    d = code.shape[-1] * 2
    shape = (8, d // 64, 4) if values else (4, d // 32, 4)
    code = code.unflatten(-1, shape).transpose(-3, -2).flatten(-3)
    n = torch.stack([code & 15, code >> 4], -1).flatten(-2).unflatten(-1, (-1, GROUP)).to(dtype)
    p = par.contiguous().view(torch.bfloat16).unflatten(-1, (-1, 2)).to(dtype)
    return (p[..., 1:] + p[..., :1] * n).flatten(-2)


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case=case)
    if case["op"] == "rotary":
        B, N, d = case["batch"], case["tokens"], case["d"]
        H, G = case["heads"], case["kv_heads"]
        dtype = getattr(torch, case["dtype"])
        if case["packed"]:  # slices of one projection of packed tokens
            x = _normal(g, N, (H + 2 * G) * d, dtype=dtype)
            st["q"] = x[:, :H * d].unflatten(-1, (H, d)).transpose(0, 1)[None]
            st["k"] = x[:, H * d:(H + G) * d].unflatten(-1, (G, d)).transpose(0, 1)[None]
            st["positions"] = torch.randint(0, case["reach"], (N,), generator=g, device="cuda", dtype=torch.int32)
        else:
            st["q"], st["k"] = _normal(g, B, H, N, d, dtype=dtype), _normal(g, B, G, N, d, dtype=dtype)
            st["positions"] = torch.arange(case["reach"] - N, case["reach"], device="cuda", dtype=torch.int32)
        st["inv_freq"], st["amplitude"] = _frequencies(case["rot"], case["factor"])
        return st
    if case["op"] == "plan":
        R, ps, W = case["requests"], case["page"], case["table"]
        old = _ragged(R, case["held_lo"], case["held_hi"])
        new = [n + 1 for n in old]
        for b in range(R):
            if case["prompt_every"] and b % case["prompt_every"] == 0:
                new[b] = min(old[b] + case["prompt"], ps * W)
            if case["shrink_every"] and b % case["shrink_every"] == 1:
                new[b] = 0 if b % 2 else old[b] // 2
        held = [-(-n // ps) for n in old]
        need = sum(max(0, -(-n // ps) - h) for n, h in zip(new, held))
        P = sum(held) + need + 13
        order = torch.randperm(P, generator=g, device="cuda", dtype=torch.int32)
        at = torch.tensor([0] + held).cumsum(0)[:-1]
        j = torch.arange(W)
        place = (at[:, None] + j).clamp(max=P - 1).cuda()
        st["table"] = torch.where((j < torch.tensor(held)[:, None]).cuda(), order[place], -1)
        # the ring of free pages, somewhere on its way round
        head = 5 * P + P // 3
        free = torch.full((P,), -1, device="cuda", dtype=torch.int32)
        count = P - sum(held)
        free[(head + torch.arange(count, device="cuda")) % P] = order[sum(held):]
        st["free"] = free
        st["free_range"] = torch.tensor([head, head + count], device="cuda")
        st["old"] = torch.tensor(old, dtype=torch.int32, device="cuda")
        st["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        st["room"] = sum(max(0, n - o) for n, o in zip(new, old)) + 3  # a padded batch
        return st
    if case["op"] == "store":
        T, G, d, ps = case["tokens"], case["kv_heads"], case["d"], case["page"]
        x = _normal(g, T, (2 * G + G) * d)
        spread = torch.exp(0.5 * torch.randn(G * d, generator=g, device="cuda"))  # channels of unlike size
        x[:, G * d:2 * G * d] *= spread.bfloat16()
        st["k"] = x[:, G * d:2 * G * d].unflatten(-1, (G, d))
        st["v"] = x[:, 2 * G * d:].unflatten(-1, (G, d))
        t = torch.arange(T, device="cuda")
        if case["scattered"]:  # a token in a page of its own
            page = torch.randperm(T + 3, generator=g, device="cuda")
            off = torch.randint(0, ps, (T,), generator=g, device="cuda")
            st["slots"] = page[:T] * ps + off
        else:
            page = torch.randperm(-(-T // ps) + 3, generator=g, device="cuda")
            st["slots"] = page[t // ps] * ps + t % ps
        st["cache"] = torch.zeros((page.numel(), G, ps // 16, 18 * d), dtype=torch.uint8, device="cuda")
        return st
    R, G, d, ps = case["requests"], case["kv_heads"], case["d"], case["page"]
    lens, T = _lens(case), case["requests"] * case["new"]
    W = -(-max(lens) // ps) + 1
    P = sum(-(-n // ps) for n in lens) + 2
    cache = torch.empty((P, G, ps // 16, 18 * d), dtype=torch.uint8, device="cuda")
    spread = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    step = max(1, (1 << 24) // (G * ps * d))
    for at in range(0, P, step):  # filled a piece at a time
        part = cache[at:at + step]
        for i, values in ((0, False), (2, True)):
            x = torch.randn((part.shape[0], G, ps // 16, 16, d), generator=g, device="cuda")
            code, par = _rows((x if values else x * spread).bfloat16(), values)
            parts = _parts(part, d)
            parts[i].copy_(code)
            parts[i + 1].copy_(par)
    held = torch.tensor([-(-n // ps) for n in lens])
    order = torch.randperm(P, generator=g, device="cuda", dtype=torch.int32)
    j = torch.arange(W)
    place = ((held.cumsum(0) - held)[:, None] + j).clamp(max=P - 1).cuda()
    st["table"] = torch.where((j < held[:, None]).cuda(), order[place], -1)
    st["cache"] = cache
    st["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["cu_tokens"] = torch.arange(R + 1, dtype=torch.int32, device="cuda") * case["new"]
    st["q"] = _normal(g, T, case["heads"], d)
    st["most"] = case["new"]
    return st


def _lens(case):
    return _ragged(case["requests"], case["len_lo"], case["len_hi"])


# ------------------------------------------------------------------ one pass
def run(state):
    return {"rotary": _rotary, "plan": _plan, "store": _store, "attend": _attend}[state["case"]["op"]](state)


def _rotary(st):
    case = st["case"]
    backward, beside = case["direction"] == "backward", case["pairs"] == "interleaved"
    if own:
        from exact_attention_117_b200 import fa
        call = fa.rotary_backward if backward else fa.rotary
        return call(st["q"], st["k"], st["positions"], st["inv_freq"], interleaved=beside, amplitude=st["amplitude"])
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    c, s = (torch.cos(angle) * st["amplitude"]).float(), (torch.sin(angle) * st["amplitude"]).float()
    s = -s if backward else s
    return tuple(_turned(x, c, s, case["rot"], beside) for x in (st["q"], st["k"]))


def _turned(x, c, s, rot, beside):
    x32 = x.float()
    if beside:
        a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
    else:
        a, b = x32[..., :rot // 2], x32[..., rot // 2:rot]
    a, b = a * c - b * s, b * c + a * s
    y = torch.stack([a, b], -1).flatten(-2) if beside else torch.cat([a, b], -1)
    return torch.cat([y, x32[..., rot:]], -1).to(x.dtype)


def _plan(st):
    ps, T = st["case"]["page"], st["room"]
    if own:
        from exact_attention_117_b200 import fa
        p = fa.kv4_plan(st["old"], st["new"], st["table"], st["free"], st["free_range"], page_size=ps, max_tokens=T)
        return dict(lengths=p.lengths, cu_tokens=p.cu_tokens, slots=p.slots, positions=p.positions, status=p.status,
                    free_range=p.free_range, table=st["table"], free=st["free"])
    old, new, table, free = st["old"].long(), st["new"].long(), st["table"], st["free"]
    W, P = table.shape[1], free.numel()
    head, tail = st["free_range"].unbind()
    bad = ((old < 0) | (new < 0) | (old > W * ps) | (new > W * ps)).any()
    held, wanted = (old + ps - 1) // ps, (new + ps - 1) // ps
    grow, need, back = (new - old).clamp_min(0), (wanted - held).clamp_min(0), (held - wanted).clamp_min(0)
    status = (need.sum() > tail - head) * 1 + (grow.sum() > T) * 2 + bad * 4
    ok = status == 0
    grow, need, back = grow * ok, need * ok, back * ok
    cu = torch.cat([torch.zeros_like(grow[:1]), grow.cumsum(0)])
    first, given = need.cumsum(0) - need, back.cumsum(0) - back
    w = torch.arange(W, device=old.device)
    fresh = (w >= held[:, None]) & (w < (held + need)[:, None])
    popped = free[(head + first[:, None] + w - held[:, None]) % P]
    table_now = torch.where(fresh, popped, table)
    ended = (w >= wanted[:, None]) & (w < (wanted + back)[:, None])
    place = torch.where(ended, (tail + given[:, None] + w - wanted[:, None]) % P, P)
    free_now = torch.cat([free, free[:1]]).scatter(0, place.flatten(), table.flatten())[:P]
    t = torch.arange(T, device=old.device)
    r = torch.searchsorted(cu[1:], t, right=True).clamp_max(old.numel() - 1)
    pos = old[r] + t - cu[r]
    there = t < cu[-1]
    page = table_now[r, (pos // ps).clamp(0, W - 1)].long()
    slots = torch.where(there, page * ps + pos % ps, -1)
    table.copy_(table_now)
    free.copy_(free_now)
    return dict(lengths=torch.where(ok, new, old).int(), cu_tokens=cu.int(), slots=slots,
                positions=torch.where(there, pos, 0).int(), status=status.int().reshape(1),
                free_range=torch.stack([head + need.sum(), tail + back.sum()]), table=table, free=free)


def _store(st):
    k, v, cache, slots = st["k"], st["v"], st["cache"], st["slots"]
    if own:
        from exact_attention_117_b200 import fa
        fa.kv4_append(k, v, cache, slots)
        return fa.kv4_gather(cache, slots)
    d, ps = k.shape[-1], st["case"]["page"]
    page, block, row = slots // ps, slots % ps // 16, slots % 16
    parts = _parts(cache, d)
    for part, rows in zip(parts, _rows(k, False) + _rows(v, True)):
        part[page, :, block, row] = rows
    kc, kp, vc, vp = (part[page, :, block, row] for part in parts)
    return _values(kc, kp, False).bfloat16(), _values(vc, vp, True).bfloat16()


def _attend(st):
    case, q, table = st["case"], st["q"], st["table"]
    if own:
        from exact_attention_117_b200 import fa
        return fa.kv4_attention(q, st["cache"], table, st["lengths"], st["cu_tokens"], max_tokens=st["most"],
                                causal=case["causal"])
    R, new, H, G, d = case["requests"], st["most"], case["heads"], case["kv_heads"], case["d"]
    kc, kp, vc, vp = (p[table.clamp_min(0)].transpose(1, 2).flatten(2, 4) for p in _parts(st["cache"], d))
    n = st["lengths"].long()[:, None]
    x = q.float().view(R, new, G, H // G, d).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [R, G, rows, d]
    score = x @ _values(kc, kp, False).transpose(-1, -2) / math.sqrt(d)
    j = torch.arange(score.shape[-1], device=q.device)
    at = torch.arange(new, device=q.device).repeat_interleave(H // G)
    last = (n - new + at if case["causal"] else n - 1 + 0 * at)[:, None, :, None]
    score = score.masked_fill(j > last, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.clamp_min(-3e38))
    total = p.sum(-1, keepdim=True)
    o = (p @ _values(vc, vp, True)) / total.clamp_min(1e-30)
    lse = top + torch.log(total)
    o, lse = (y.unflatten(2, (new, H // G)).transpose(1, 2).reshape(R * new, H, -1) for y in (o, lse))
    return o.to(q.dtype), lse[..., 0].contiguous()


# ------------------------------------------------------------------ the least work
def work(case):
    if case["op"] == "rotary":
        el = case["batch"] * (case["heads"] + case["kv_heads"]) * case["tokens"] * case["d"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": 2 * el * size + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * el * case["rot"] // case["d"]}
    if case["op"] == "plan":
        R, ps, W = case["requests"], case["page"], case["table"]
        old = _ragged(R, case["held_lo"], case["held_hi"])
        tokens = pages = 0
        for b in range(R):
            new = old[b] + 1
            if case["prompt_every"] and b % case["prompt_every"] == 0:
                new = min(old[b] + case["prompt"], ps * W)
            if case["shrink_every"] and b % case["shrink_every"] == 1:
                new = 0 if b % 2 else old[b] // 2
            tokens += max(0, new - old[b])
            pages += abs(-(-new // ps) - -(-old[b] // ps))
        return {"bytes": 16 * R + 12 * (tokens + 3) + 8 * pages + 36, "flops": 0}
    if case["op"] == "store":
        el = case["tokens"] * case["kv_heads"] * case["d"]
        return {"bytes": 2 * el * (4 + 1.125) + 16 * case["tokens"], "flops": 2 * el * 8}
    lens, new, d = _lens(case), case["new"], case["d"]
    seen = sum(new * n - new * (new - 1) // 2 if case["causal"] else new * n for n in lens)
    rows = case["requests"] * new * case["heads"]
    return {"bytes": sum(lens) * case["kv_heads"] * d * 1.125 + rows * (4 * d + 4) + sum(lens) // case["page"] * 4,
            "flops": 4 * d * case["heads"] * seen}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "plan":
        return None  # whole numbers only
    if case["op"] == "rotary":
        sign = -1.0 if case["direction"] == "backward" else 1.0
        turn = torch.polar(torch.full((), st["amplitude"], dtype=torch.float64, device="cuda"),
                           sign * st["positions"].double()[:, None] * st["inv_freq"])
        out = []
        for x in (st["q"], st["k"]):
            y, rot = x.double().clone(), case["rot"]
            first, second = ((slice(0, rot, 2), slice(1, rot, 2)) if case["pairs"] == "interleaved"
                             else (slice(0, rot // 2), slice(rot // 2, rot)))
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
        return tuple(out)
    if case["op"] == "store":
        out = []
        for x in (st["k"], st["v"]):
            x = x.double()
            y = torch.empty_like(x)
            for c in range(0, x.shape[-1], GROUP):
                z = x[..., c:c + GROUP]
                lo, hi = z.min(-1, keepdim=True).values, z.max(-1, keepdim=True).values
                want = (hi - lo) / 15.0
                # the next value of eight significant bits at or above
                unit = torch.exp2((torch.frexp(want.clamp_min(1e-30)).exponent - 8).double())
                scale = torch.ceil(want / unit) * unit
                steps = torch.floor((z - lo) / scale.clamp_min(1e-30) + 0.5).clamp(0.0, 15.0)
                y[..., c:c + GROUP] = torch.where(scale > 0, lo + steps * scale, lo)
            out.append(y)
        return tuple(out)
    H, G, d, new, ps = case["heads"], case["kv_heads"], case["d"], case["new"], case["page"]
    o = torch.empty((case["requests"] * new, H, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((case["requests"] * new, H), dtype=torch.float64, device="cuda")
    # places of each channel's code in a row, as half bytes
    word = torch.arange(d) // 8
    at = [((word % 4) * (d // 32) + word // 4) * 8 + torch.arange(d) % 8, ((word % 8) * (d // 64) + word // 8) * 8 + torch.arange(d) % 8]
    for b, n in enumerate(_lens(case)):
        tiles = st["cache"][st["table"][b, :-(-n // ps)].long()].transpose(0, 1).flatten(1, 2)  # [G, blocks, bytes]
        for h in range(G):
            kv = []
            for i in range(2):
                t = tiles[h, :, i * 9 * d:(i + 1) * 9 * d]
                code = t[:, :8 * d].reshape(-1, d // 2).int()
                half = torch.stack([code % 16, code // 16], 2).flatten(1)[:n, at[i].cuda()].double()
                par = t[:, 8 * d:].contiguous().view(torch.bfloat16).view(-1, d // 64, 2)[:n].double()
                par = par.repeat_interleave(GROUP, 1)
                kv.append(par[..., 1] + par[..., 0] * half)
            for r in range(h * (H // G), (h + 1) * (H // G)):
                s = st["q"][b * new:(b + 1) * new, r].double() @ kv[0].T * d ** -0.5
                if case["causal"]:
                    s += torch.full_like(s, -math.inf).triu(n - new + 1)
                lse[b * new:(b + 1) * new, r] = torch.logsumexp(s, 1)
                o[b * new:(b + 1) * new, r] = torch.softmax(s, 1) @ kv[1]
    return o, lse
